// api.cu -- the C ABI declared in include/gemma_attn.h: host-side validation, owner-layer
// resolution, the split plan of the decode bucket, and kernel launches. Nothing here
// allocates memory or synchronises; every launch goes to the caller's stream.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/gemma_attn.h"
#include "attn_internal.h"
#include "logits.h"
#include "q4.h"
#include "sample.h"
#include "tree.h"

using gemma::RowsParams;

namespace {

constexpr int kMaxSplit = 128;
#ifndef GEMMA_MIN_CHUNK_KEYS
#define GEMMA_MIN_CHUNK_KEYS 256
#endif
#ifndef GEMMA_SPLIT_CTAS_PER_SM
#define GEMMA_SPLIT_CTAS_PER_SM 8
#endif
constexpr int kMinChunkKeys = GEMMA_MIN_CHUNK_KEYS;  // keys per split chunk when work is plentiful
// no split when the (sequence, KV head) units alone fill the GPU (at least this many per SM)
// and each attends a short key range: one CTA per unit, no partials, no combine launch
constexpr long long kNoSplitUnitsPerSm = 2;
constexpr long long kNoSplitMaxKeys = 2048;
constexpr long long kSplitCtasPerSm = GEMMA_SPLIT_CTAS_PER_SM;

// SM count of the current device, cached per device (atomics: calls may come from several
// host threads; they all store the same value)
int sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return -1;
    if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }
bool group_ok(int g) { return g == 1 || g == 2 || g == 4 || g == 8 || g == 16; }
long long round_up(long long x, long long m) { return (x + m - 1) / m * m; }

int check_shape(int kind, int window, int n_q, int n_kv, int head_dim, int dtype) {
    if (kind != GEMMA_SLIDING && kind != GEMMA_GLOBAL && kind != GEMMA_SLIDING_RING)
        return GEMMA_ERR_INVALID_ARG;
    if (kind != GEMMA_GLOBAL && window < 1) return GEMMA_ERR_INVALID_ARG;
    if (n_q < 1 || n_kv < 1 || n_q % n_kv != 0) return GEMMA_ERR_INVALID_ARG;
    if (dtype != GEMMA_BF16 && dtype != GEMMA_FP32) return GEMMA_ERR_INVALID_ARG;
    if (!head_dim_ok(head_dim) || !group_ok(n_q / n_kv)) return GEMMA_ERR_UNSUPPORTED;
    return GEMMA_OK;
}

// Owner resolution ("Porting Gemma-4 (2B / 4B / 12B) to AWS Inferentia2", section 2.1): a
// layer reads the cache of owner_map[layer], an earlier layer that owns its cache.
int resolve_owner(const int32_t* owner_map, int n_layers, int layer, int* owner) {
    if (!owner_map || n_layers < 1 || layer < 0 || layer >= n_layers) return GEMMA_ERR_INVALID_ARG;
    const int o = owner_map[layer];
    if (o < 0 || o > layer || owner_map[o] != o) return GEMMA_ERR_INVALID_ARG;
    *owner = o;
    return GEMMA_OK;
}

struct Plan {
    int n_split;
    int chunk;
    size_t o_bytes;   // partial outputs
    size_t ws_bytes;  // total scratch
    int cluster;      // the chunks of a row tile merge inside their cluster (no scratch)
};

// Splits of at most this many chunks run as one thread-block cluster per (sequence, KV head)
// and merge through distributed shared memory; plans of up to twice as many chunks are
// coarsened to it (one launch and no scratch beat twice the CTAs plus a combine pass). When all
// CTAs of a plan of up to kMaxBigClusterSplit chunks fit on the GPU at once (one per SM), a
// latency-bound small batch, the plan keeps its chunks and runs as clusters of that many (above
// the portable cluster size; fewer keys per CTA matter more there than the wider merge).
constexpr int kMaxClusterSplit = 8;
constexpr int kMaxBigClusterSplit = 16;
// A latency-bound plan finer than the largest cluster is coarsened to one cluster of
// kMaxBigClusterSplit chunks (no combine launch) while each chunk stays at most this many keys
// (a few key tiles per CTA; longer chunks cost more per CTA than the combine pass saves).
constexpr long long kBigClusterMaxKeys = 128;

// Decode splits each (sequence, KV head) key range into chunks so that enough CTAs stream
// the cache at once: about one chunk per SM for small problems, about eight per SM (and at
// least kMinChunkKeys keys each) for large ones; not at all when the units alone fill the GPU
// over short key ranges (a sliding window across a large batch). Prefill has one row tile per 16 rows and no
// split. Depends only on the arguments and the SM count.
Plan make_plan(int batch, int kind, int window, int n_q, int n_kv, int head_dim, int max_seq_len,
               int n_tok, int n_sm, bool paged = false) {
    Plan pl{1, 1 << 30, 0, 0, 0};
    if (n_tok != 1) return pl;
    const long long T = gemma::kKeyTile;
    long long n_read = kind != GEMMA_GLOBAL && window < max_seq_len ? window : max_seq_len;
    // a ring cache's or paged pool's key tiles start at multiples of the tile (so that none wraps
    // or crosses a page): up to T - 1 keys before the window join the range
    if (kind == GEMMA_SLIDING_RING || paged) n_read += T - 1;
    if ((long long)batch * n_kv >= kNoSplitUnitsPerSm * n_sm && n_read <= kNoSplitMaxKeys) return pl;
    const long long total = (long long)batch * n_kv * n_read;
    const long long one_per_sm = round_up((total + n_sm - 1) / n_sm, T);
    const long long eight_per_sm =
        round_up((total + kSplitCtasPerSm * n_sm - 1) / (kSplitCtasPerSm * n_sm), T);
    long long chunk = one_per_sm < kMinChunkKeys ? one_per_sm : kMinChunkKeys;
    if (eight_per_sm > chunk) chunk = eight_per_sm;
    if (chunk < T) chunk = T;
    long long n_split = (n_read + chunk - 1) / chunk;
    if (n_split > kMaxSplit) {
        chunk = round_up((n_read + kMaxSplit - 1) / kMaxSplit, T);
        n_split = (n_read + chunk - 1) / chunk;
    }
    if (n_split <= 1) return pl;
    if (n_split <= kMaxBigClusterSplit && (long long)batch * n_kv * n_split <= n_sm) {
        pl.n_split = (int)n_split;
        pl.chunk = (int)chunk;
        pl.cluster = 1;
        return pl;
    }
    if (n_split > kMaxBigClusterSplit && (long long)batch * n_kv * kMaxBigClusterSplit <= n_sm &&
        n_read <= kMaxBigClusterSplit * kBigClusterMaxKeys) {
        chunk = round_up((n_read + kMaxBigClusterSplit - 1) / kMaxBigClusterSplit, T);
        n_split = (n_read + chunk - 1) / chunk;
        pl.n_split = (int)n_split;
        pl.chunk = (int)chunk;
        pl.cluster = 1;
        return pl;
    }
    if (n_split <= 2 * kMaxClusterSplit) {
        if (n_split > kMaxClusterSplit) {
            chunk = round_up((n_read + kMaxClusterSplit - 1) / kMaxClusterSplit, T);
            n_split = (n_read + chunk - 1) / chunk;
        }
        pl.n_split = (int)n_split;
        pl.chunk = (int)chunk;
        pl.cluster = 1;
        return pl;
    }
    pl.n_split = (int)n_split;
    pl.chunk = (int)chunk;
    const size_t rows = (size_t)batch * n_q * n_split;
    pl.o_bytes = (size_t)round_up((long long)(rows * head_dim * sizeof(float)), 256);
    pl.ws_bytes = pl.o_bytes + (size_t)round_up((long long)(rows * 2 * sizeof(float)), 256);
    return pl;
}

int attention(void* out, const void* q, const void* const* k_cache, const void* const* v_cache,
              const int32_t* owner_map, int n_layers, int layer, const int32_t* seq_lens,
              int max_seq_len, int n_tok, int batch, int kind, int window, int n_q, int n_kv,
              int head_dim, int k_eq_v, int kv_capacity, float scale, float softcap, int dtype,
              void* workspace, size_t workspace_bytes, uint32_t* device_error, void* stream,
              const int32_t* n_real = nullptr, const void* k_new = nullptr,
              const void* v_new = nullptr, const int32_t* write_pos = nullptr,
              const gemma::PagedLayout* pg = nullptr) {
    if (batch < 0 || n_tok < 1) return GEMMA_ERR_INVALID_ARG;
    if (pg) {  // paged pool: a multiple of 128 keys per page, so that no key tile crosses a page
        if (kind == GEMMA_SLIDING_RING || pg->page_size < 128 || pg->page_size % 128 != 0 ||
            pg->max_pages < 1 || pg->n_pages < 1)
            return pg->page_size > 0 && pg->page_size % 128 != 0 ? GEMMA_ERR_UNSUPPORTED
                                                                  : GEMMA_ERR_INVALID_ARG;
        if ((long long)pg->max_pages * pg->page_size > (1ll << 30) ||
            (long long)pg->n_pages * n_kv > (1ll << 31) - 1)
            return GEMMA_ERR_UNSUPPORTED;
        if (batch > 0 && !pg->block_table) return GEMMA_ERR_INVALID_ARG;
        kv_capacity = pg->max_pages * pg->page_size;  // logical capacity of a sequence
    }
    if (!std::isfinite(softcap) || softcap < 0.f) return GEMMA_ERR_INVALID_ARG;
    int st = check_shape(kind, window, n_q, n_kv, head_dim, dtype);
    if (st != GEMMA_OK) return st;
    int o = 0;
    st = resolve_owner(owner_map, n_layers, layer, &o);
    if (st != GEMMA_OK) return st;
    if (kv_capacity < 1 || max_seq_len < n_tok || !std::isfinite(scale) || !(scale > 0.f))
        return GEMMA_ERR_INVALID_ARG;
    const bool ring = kind == GEMMA_SLIDING_RING;
    if (ring) {
        if (kv_capacity % 128 != 0) return GEMMA_ERR_UNSUPPORTED;
        if ((long long)kv_capacity < (long long)window + n_tok - 1) return GEMMA_ERR_CAPACITY;
    } else if (max_seq_len > kv_capacity) {
        return GEMMA_ERR_CAPACITY;
    }
    if (batch > 65535) return GEMMA_ERR_UNSUPPORTED;
    if (batch == 0) return GEMMA_OK;
    if (!out || !q || !seq_lens || !k_cache || !k_cache[o]) return GEMMA_ERR_INVALID_ARG;
    const void* kc = k_cache[o];
    const void* vc = kc;
    if (!k_eq_v) {
        if (!v_cache || !v_cache[o]) return GEMMA_ERR_INVALID_ARG;
        vc = v_cache[o];
    }
    if (!aligned16(out) || !aligned16(q) || !aligned16(kc) || !aligned16(vc))
        return GEMMA_ERR_INVALID_ARG;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    // a padded bucket is never split over keys (pad rows have no key range to merge)
    Plan pl = n_real ? Plan{1, 1 << 30, 0, 0, 0}
                           : make_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len,
                                       n_tok, n_sm, pg != nullptr);
    if (pl.ws_bytes > 0 &&
        (!workspace || workspace_bytes < pl.ws_bytes || !aligned16(workspace)))
        return GEMMA_ERR_WORKSPACE;

    RowsParams p{};
    p.q = q;
    p.k = kc;
    p.v = vc;
    p.seq_lens = seq_lens;
    p.n_real = n_real;
    p.k_new = k_new;
    p.v_new = v_new;
    p.write_pos = write_pos;
    p.out = out;
    p.o_part = pl.ws_bytes ? static_cast<float*>(workspace) : nullptr;
    p.ml_part = pl.ws_bytes
                    ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.o_bytes)
                    : nullptr;
    p.err = device_error;
    p.n_tok = n_tok;
    p.n_q = n_q;
    p.n_kv = n_kv;
    p.G = n_q / n_kv;
    p.cap = kv_capacity;
    p.window = window;
    p.is_sliding = kind != GEMMA_GLOBAL;
    p.ring = ring ? kv_capacity : 0;
    if (pg) {
        p.block_table = pg->block_table;
        p.page_size = pg->page_size;
        p.max_pages = pg->max_pages;
        p.n_pages = pg->n_pages;
    }
    p.k_eq_v = k_eq_v ? 1 : 0;
    p.max_seq_len = max_seq_len;
    if (pl.cluster && dtype != GEMMA_BF16) {
        // the fp32 debug path does not split a clustered plan: one pass per row
        pl.n_split = 1;
        pl.chunk = 1 << 30;
        pl.cluster = 0;
    }
    p.n_split = pl.n_split;
    p.chunk = pl.chunk;
    p.cluster = pl.cluster;
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.softcap = softcap;
    p.cap_inner = softcap > 0.f ? scale / softcap : 0.f;
    p.cap_log2 = softcap * 1.4426950408889634f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long rows = (long long)n_tok * p.G;
    cudaError_t e;
    if (dtype == GEMMA_BF16 && (n_tok > 1 || n_real) && gemma::prefill_tc_supported(head_dim)) {
        e = gemma::launch_prefill_tc(p, head_dim, batch, s);
    } else if (dtype == GEMMA_BF16) {
        const size_t smem = gemma::rows_bf16_smem_bytes(head_dim, p.k_eq_v, &p.n_stages);
        const long long tiles = (rows + gemma::kRowTile - 1) / gemma::kRowTile;
        e = gemma::launch_rows_bf16(p, head_dim, dim3((unsigned)(tiles * pl.n_split), n_kv, batch),
                                    smem, s);
    } else {
        const long long tiles = (rows + gemma::kF32RowsPerCta - 1) / gemma::kF32RowsPerCta;
        e = gemma::launch_rows_f32(p, head_dim, dim3((unsigned)(tiles * pl.n_split), n_kv, batch),
                                   s);
    }
    if (e == cudaSuccess && pl.n_split > 1 && !pl.cluster)
        e = gemma::launch_combine(p, head_dim, batch, dtype == GEMMA_FP32, s);
    return e == cudaSuccess ? GEMMA_OK : GEMMA_ERR_CUDA;
}

int append_rows(void* const* k_cache, void* const* v_cache, const int32_t* owner_map,
                int n_layers, int layer, const void* k_new, const void* v_new,
                const int32_t* write_pos, const int32_t* n_real, int ring, int batch, int n_new,
                int n_kv, int head_dim, int kv_capacity, int k_eq_v, gemma_dtype dtype,
                uint32_t* device_error, void* stream,
                const gemma::PagedLayout& pg = gemma::PagedLayout{nullptr, 0, 0, 0});

}  // namespace

extern "C" {

int gemma_abi_version(void) { return 1; }

const char* gemma_status_string(int status) {
    switch (status) {
        case GEMMA_OK: return "GEMMA_OK";
        case GEMMA_ERR_INVALID_ARG: return "GEMMA_ERR_INVALID_ARG";
        case GEMMA_ERR_UNSUPPORTED: return "GEMMA_ERR_UNSUPPORTED";
        case GEMMA_ERR_CAPACITY: return "GEMMA_ERR_CAPACITY";
        case GEMMA_ERR_WORKSPACE: return "GEMMA_ERR_WORKSPACE";
        case GEMMA_ERR_CUDA: return "GEMMA_ERR_CUDA";
    }
    return "GEMMA_UNKNOWN_STATUS";
}

int gemma_kv_append(void* const* k_cache, void* const* v_cache, const int32_t* owner_map,
                    int n_layers, int layer, const void* k_new, const void* v_new,
                    const int32_t* write_pos, int batch, int n_new, int n_kv, int head_dim,
                    int kv_capacity, int k_eq_v, gemma_dtype dtype, uint32_t* device_error,
                    void* stream) {
    return append_rows(k_cache, v_cache, owner_map, n_layers, layer, k_new, v_new, write_pos,
                       nullptr, 0, batch, n_new, n_kv, head_dim, kv_capacity, k_eq_v, dtype,
                       device_error, stream);
}

int gemma_kv_append_ring(void* const* k_cache, void* const* v_cache, const int32_t* owner_map,
                         int n_layers, int layer, const void* k_new, const void* v_new,
                         const int32_t* write_pos, int batch, int n_new, int n_kv, int head_dim,
                         int kv_capacity, int k_eq_v, gemma_dtype dtype, uint32_t* device_error,
                         void* stream) {
    return append_rows(k_cache, v_cache, owner_map, n_layers, layer, k_new, v_new, write_pos,
                       nullptr, kv_capacity, batch, n_new, n_kv, head_dim, kv_capacity, k_eq_v,
                       dtype, device_error, stream);
}

int gemma_kv_append_bucket(void* const* k_cache, void* const* v_cache, const int32_t* owner_map,
                           int n_layers, int layer, const void* k_new, const void* v_new,
                           const int32_t* write_pos, const int32_t* n_real, int batch, int n_new,
                           int n_kv, int head_dim, int kv_capacity, int k_eq_v, gemma_dtype dtype,
                           uint32_t* device_error, void* stream) {
    if (!n_real && batch > 0 && n_new > 0) return GEMMA_ERR_INVALID_ARG;
    return append_rows(k_cache, v_cache, owner_map, n_layers, layer, k_new, v_new, write_pos,
                       n_real, 0, batch, n_new, n_kv, head_dim, kv_capacity, k_eq_v, dtype,
                       device_error, stream);
}

}  // extern "C"

namespace {

int append_rows(void* const* k_cache, void* const* v_cache, const int32_t* owner_map,
                int n_layers, int layer, const void* k_new, const void* v_new,
                const int32_t* write_pos, const int32_t* n_real, int ring, int batch, int n_new,
                int n_kv, int head_dim, int kv_capacity, int k_eq_v, gemma_dtype dtype,
                uint32_t* device_error, void* stream, const gemma::PagedLayout& pg) {
    if (batch < 0 || n_new < 0 || n_kv < 1 || kv_capacity < 1) return GEMMA_ERR_INVALID_ARG;
    if (dtype != GEMMA_BF16 && dtype != GEMMA_FP32) return GEMMA_ERR_INVALID_ARG;
    if (!head_dim_ok(head_dim)) return GEMMA_ERR_UNSUPPORTED;
    int o = 0;
    int st = resolve_owner(owner_map, n_layers, layer, &o);
    if (st != GEMMA_OK) return st;
    if (o != layer) return GEMMA_OK;  // a shared layer writes no cache
    if (n_new > kv_capacity) return GEMMA_ERR_CAPACITY;
    if (batch == 0 || n_new == 0) return GEMMA_OK;
    if (!k_cache || !k_cache[layer] || !k_new || !write_pos) return GEMMA_ERR_INVALID_ARG;
    void* vc = nullptr;
    if (!k_eq_v) {
        if (!v_cache || !v_cache[layer] || !v_new) return GEMMA_ERR_INVALID_ARG;
        vc = v_cache[layer];
    }
    if (!aligned16(k_cache[layer]) || !aligned16(k_new) ||
        (vc && (!aligned16(vc) || !aligned16(v_new))))
        return GEMMA_ERR_INVALID_ARG;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    const int row_bytes = head_dim * (dtype == GEMMA_BF16 ? 2 : 4);
    cudaError_t e = gemma::launch_kv_append(k_cache[layer], vc, k_new, vc ? v_new : nullptr,
                                            write_pos, n_real, ring, pg, batch, n_new, n_kv,
                                            kv_capacity,
                                            row_bytes, device_error, n_sm,
                                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMMA_OK : GEMMA_ERR_CUDA;
}

}  // namespace

extern "C" {

int gemma_attn_decode(void* out, const void* q, const void* const* k_cache,
                      const void* const* v_cache, const int32_t* owner_map, int n_layers,
                      int layer, const int32_t* seq_lens, int max_seq_len, int batch,
                      gemma_layer_kind kind, int window, int n_q, int n_kv, int head_dim,
                      int k_eq_v, int kv_capacity, float scale, gemma_dtype dtype,
                      void* workspace, size_t workspace_bytes, uint32_t* device_error,
                      void* stream) {
    return attention(out, q, k_cache, v_cache, owner_map, n_layers, layer, seq_lens, max_seq_len,
                     1, batch, kind, window, n_q, n_kv, head_dim, k_eq_v, kv_capacity, scale, 0.f,
                     dtype, workspace, workspace_bytes, device_error, stream);
}

int gemma_attn_prefill(void* out, const void* q, const void* const* k_cache,
                       const void* const* v_cache, const int32_t* owner_map, int n_layers,
                       int layer, const int32_t* seq_lens, int max_seq_len, int n_new,
                       int batch, gemma_layer_kind kind, int window, int n_q, int n_kv,
                       int head_dim, int k_eq_v, int kv_capacity, float scale,
                       gemma_dtype dtype, void* workspace, size_t workspace_bytes,
                       uint32_t* device_error, void* stream) {
    if (n_new == 0 && batch >= 0) return GEMMA_OK;
    return attention(out, q, k_cache, v_cache, owner_map, n_layers, layer, seq_lens, max_seq_len,
                     n_new, batch, kind, window, n_q, n_kv, head_dim, k_eq_v, kv_capacity, scale,
                     0.f, dtype, workspace, workspace_bytes, device_error, stream);
}

int gemma_attn_softcap(void* out, const void* q, const void* const* k_cache,
                       const void* const* v_cache, const int32_t* owner_map, int n_layers,
                       int layer, const int32_t* seq_lens, int max_seq_len, int n_new,
                       int batch, gemma_layer_kind kind, int window, int n_q, int n_kv,
                       int head_dim, int k_eq_v, int kv_capacity, float scale, float softcap,
                       gemma_dtype dtype, void* workspace, size_t workspace_bytes,
                       uint32_t* device_error, void* stream) {
    if (n_new == 0 && batch >= 0) return GEMMA_OK;
    return attention(out, q, k_cache, v_cache, owner_map, n_layers, layer, seq_lens, max_seq_len,
                     n_new, batch, kind, window, n_q, n_kv, head_dim, k_eq_v, kv_capacity, scale,
                     softcap, dtype, workspace, workspace_bytes, device_error, stream);
}

int gemma_attn_decode_append(void* out, const void* q, void* const* k_cache, void* const* v_cache,
                             const int32_t* owner_map, int n_layers, int layer, const void* k_new,
                             const void* v_new, const int32_t* write_pos,
                             const int32_t* seq_lens, int max_seq_len, int batch,
                             gemma_layer_kind kind, int window, int n_q, int n_kv, int head_dim,
                             int k_eq_v, int kv_capacity, float scale, gemma_dtype dtype,
                             void* workspace, size_t workspace_bytes, uint32_t* device_error,
                             void* stream) {
    int o = 0;
    int st = resolve_owner(owner_map, n_layers, layer, &o);
    if (st != GEMMA_OK) return st;
    const void* const* kcc = const_cast<const void* const*>(k_cache);
    const void* const* vcc = const_cast<const void* const*>(v_cache);
    if (o != layer)  // a shared layer appends nothing: plain decode against the owner's cache
        return attention(out, q, kcc, vcc, owner_map, n_layers, layer, seq_lens, max_seq_len, 1,
                         batch, kind, window, n_q, n_kv, head_dim, k_eq_v, kv_capacity, scale,
                         0.f, dtype, workspace, workspace_bytes, device_error, stream);
    if (batch > 0 && (!k_new || !write_pos || (!k_eq_v && !v_new))) return GEMMA_ERR_INVALID_ARG;
    if (batch > 0 && (!aligned16(k_new) || (!k_eq_v && !aligned16(v_new))))
        return GEMMA_ERR_INVALID_ARG;
    if (dtype != GEMMA_BF16) {
        // the fp32 debug path keeps two launches: append, then attend
        st = append_rows(k_cache, v_cache, owner_map, n_layers, layer, k_new, v_new, write_pos,
                         nullptr, kind == GEMMA_SLIDING_RING ? kv_capacity : 0, batch, 1, n_kv,
                         head_dim, kv_capacity, k_eq_v, dtype, device_error, stream);
        if (st != GEMMA_OK) return st;
        return attention(out, q, kcc, vcc, owner_map, n_layers, layer, seq_lens, max_seq_len, 1,
                         batch, kind, window, n_q, n_kv, head_dim, k_eq_v, kv_capacity, scale,
                         0.f, dtype, workspace, workspace_bytes, device_error, stream);
    }
    return attention(out, q, kcc, vcc, owner_map, n_layers, layer, seq_lens, max_seq_len, 1, batch,
                     kind, window, n_q, n_kv, head_dim, k_eq_v, kv_capacity, scale, 0.f, dtype,
                     workspace, workspace_bytes, device_error, stream, nullptr, k_new,
                     k_eq_v ? nullptr : v_new, write_pos);
}

namespace {
int check_paged(int max_pages, int page_size, int n_pages) {
    if (page_size > 0 && page_size % 128 != 0) return GEMMA_ERR_UNSUPPORTED;
    if (page_size < 128 || max_pages < 1 || n_pages < 1) return GEMMA_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > (1ll << 30)) return GEMMA_ERR_UNSUPPORTED;
    return GEMMA_OK;
}
}  // namespace

int gemma_kv_append_paged(void* const* k_pool, void* const* v_pool, const int32_t* owner_map,
                          int n_layers, int layer, const void* k_new, const void* v_new,
                          const int32_t* write_pos, const int32_t* block_table, int max_pages,
                          int page_size, int n_pages, int batch, int n_new, int n_kv,
                          int head_dim, int k_eq_v, gemma_dtype dtype, uint32_t* device_error,
                          void* stream) {
    const int st = check_paged(max_pages, page_size, n_pages);
    if (st != GEMMA_OK) return st;
    if (batch > 0 && n_new > 0 && !block_table) return GEMMA_ERR_INVALID_ARG;
    const gemma::PagedLayout pg{block_table, max_pages, page_size, n_pages};
    return append_rows(k_pool, v_pool, owner_map, n_layers, layer, k_new, v_new, write_pos,
                       nullptr, 0, batch, n_new, n_kv, head_dim, max_pages * page_size, k_eq_v,
                       dtype, device_error, stream, pg);
}

int gemma_attn_paged(void* out, const void* q, void* const* k_pool, void* const* v_pool,
                     const int32_t* owner_map, int n_layers, int layer, const int32_t* seq_lens,
                     const int32_t* block_table, int max_pages, int page_size, int n_pages,
                     int max_seq_len, int n_new, int batch, gemma_layer_kind kind, int window,
                     int n_q, int n_kv, int head_dim, int k_eq_v, float scale, gemma_dtype dtype,
                     const void* k_new, const void* v_new, const int32_t* write_pos,
                     void* workspace, size_t workspace_bytes, uint32_t* device_error,
                     void* stream) {
    if (n_new == 0 && batch >= 0) return GEMMA_OK;
    int st = check_paged(max_pages, page_size, n_pages);
    if (st != GEMMA_OK) return st;
    const gemma::PagedLayout pg{block_table, max_pages, page_size, n_pages};
    const void* const* kcc = const_cast<const void* const*>(k_pool);
    const void* const* vcc = const_cast<const void* const*>(v_pool);
    int o = 0;
    st = resolve_owner(owner_map, n_layers, layer, &o);
    if (st != GEMMA_OK) return st;
    if (k_new && o == layer) {  // this step's rows are written by the decode launch itself
        if (n_new != 1) return GEMMA_ERR_INVALID_ARG;
        if (batch > 0 && (!write_pos || (!k_eq_v && !v_new))) return GEMMA_ERR_INVALID_ARG;
        if (batch > 0 && (!aligned16(k_new) || (!k_eq_v && !aligned16(v_new))))
            return GEMMA_ERR_INVALID_ARG;
        if (dtype != GEMMA_BF16) {  // the fp32 debug path: append, then attend
            st = append_rows(k_pool, v_pool, owner_map, n_layers, layer, k_new, v_new, write_pos,
                             nullptr, 0, batch, 1, n_kv, head_dim, max_pages * page_size, k_eq_v,
                             dtype, device_error, stream, pg);
            if (st != GEMMA_OK) return st;
        } else {
            return attention(out, q, kcc, vcc, owner_map, n_layers, layer, seq_lens, max_seq_len,
                             1, batch, kind, window, n_q, n_kv, head_dim, k_eq_v, 0, scale, 0.f,
                             dtype, workspace, workspace_bytes, device_error, stream, nullptr,
                             k_new, k_eq_v ? nullptr : v_new, write_pos, &pg);
        }
    }
    return attention(out, q, kcc, vcc, owner_map, n_layers, layer, seq_lens, max_seq_len, n_new,
                     batch, kind, window, n_q, n_kv, head_dim, k_eq_v, 0, scale, 0.f, dtype,
                     workspace, workspace_bytes, device_error, stream, nullptr, nullptr, nullptr,
                     nullptr, &pg);
}

size_t gemma_attn_workspace_size_paged(int batch, gemma_layer_kind kind, int window, int n_q,
                                       int n_kv, int head_dim, int max_seq_len, int n_new) {
    if (batch < 0 || n_new < 1 || max_seq_len < n_new || kind == GEMMA_SLIDING_RING)
        return (size_t)-1;
    if (check_shape(kind, window, n_q, n_kv, head_dim, GEMMA_BF16) != GEMMA_OK) return (size_t)-1;
    if (batch == 0) return 0;
    const int n_sm = sm_count();
    if (n_sm < 0) return (size_t)-1;
    return make_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_new, n_sm, true)
        .ws_bytes;
}

int gemma_attn_prefill_bucket(void* out, const void* q, const void* const* k_cache,
                              const void* const* v_cache, const int32_t* owner_map, int n_layers,
                              int layer, const int32_t* seq_lens, const int32_t* n_real,
                              int max_seq_len, int n_new, int batch, gemma_layer_kind kind,
                              int window, int n_q, int n_kv, int head_dim, int k_eq_v,
                              int kv_capacity, float scale, gemma_dtype dtype, void* workspace,
                              size_t workspace_bytes, uint32_t* device_error, void* stream) {
    if (n_new == 0 && batch >= 0) return GEMMA_OK;
    if (!n_real && batch > 0) return GEMMA_ERR_INVALID_ARG;
    return attention(out, q, k_cache, v_cache, owner_map, n_layers, layer, seq_lens, max_seq_len,
                     n_new, batch, kind, window, n_q, n_kv, head_dim, k_eq_v, kv_capacity, scale,
                     0.f, dtype, workspace, workspace_bytes, device_error, stream, n_real);
}

size_t gemma_attn_workspace_size(int batch, gemma_layer_kind kind, int window, int n_q,
                                 int n_kv, int head_dim, int max_seq_len, int n_new) {
    if (batch < 0 || n_new < 1 || max_seq_len < n_new) return (size_t)-1;
    if (check_shape(kind, window, n_q, n_kv, head_dim, GEMMA_BF16) != GEMMA_OK) return (size_t)-1;
    if (batch == 0) return 0;
    const int n_sm = sm_count();
    if (n_sm < 0) return (size_t)-1;
    return make_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_new, n_sm).ws_bytes;
}

int gemma_logit_softcap_argmax(const void* logits, int batch, int vocab, gemma_dtype dtype,
                               float softcap, void* capped_out, int32_t* argmax_out,
                               void* workspace, size_t workspace_bytes, void* stream) {
    if (batch < 0 || vocab < 1 || (dtype != GEMMA_BF16 && dtype != GEMMA_FP32))
        return GEMMA_ERR_INVALID_ARG;
    if (!std::isfinite(softcap) || softcap < 0.f) return GEMMA_ERR_INVALID_ARG;
    if (batch == 0) return GEMMA_OK;
    if (batch > 65535) return GEMMA_ERR_UNSUPPORTED;  // one grid row per batch row
    if (!logits || !argmax_out || !aligned16(logits) || (capped_out && !aligned16(capped_out)))
        return GEMMA_ERR_INVALID_ARG;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    const gemma::LogitPlan pl = gemma::logit_plan(batch, vocab, n_sm);
    if (pl.ws_bytes > 0 && (!workspace || workspace_bytes < pl.ws_bytes || !aligned16(workspace)))
        return GEMMA_ERR_WORKSPACE;
    const cudaError_t e = gemma::launch_logit_softcap_argmax(
        logits, capped_out, argmax_out, workspace, batch, vocab, dtype == GEMMA_FP32, softcap, pl,
        static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMMA_OK : GEMMA_ERR_CUDA;
}

size_t gemma_logit_workspace_size(int batch, int vocab) {
    if (batch < 0 || vocab < 1) return (size_t)-1;
    if (batch == 0) return 0;
    const int n_sm = sm_count();
    if (n_sm < 0) return (size_t)-1;
    return gemma::logit_plan(batch, vocab, n_sm).ws_bytes;
}

// ---------------------------------------------------------------------------------------------
// 4-bit KV cache
// ---------------------------------------------------------------------------------------------
namespace {

// Kind, layout and sizes of a 4-bit cache; fills everything of *c but the pointers.
int q4_layout(int kind, int n_kv, int head_dim, int kv_capacity, const int32_t* block_table,
              int max_pages, int page_size, int n_pages, gemma::Q4Cache* c) {
    if (kind != GEMMA_SLIDING && kind != GEMMA_GLOBAL && kind != GEMMA_SLIDING_RING)
        return GEMMA_ERR_INVALID_ARG;
    if (n_kv < 1) return GEMMA_ERR_INVALID_ARG;
    // (one grid layer per KV head, of K and of V)
    if (!head_dim_ok(head_dim) || n_kv > 32767) return GEMMA_ERR_UNSUPPORTED;
    *c = gemma::Q4Cache{};
    c->n_kv = n_kv;
    if (block_table) {
        if (kind == GEMMA_SLIDING_RING) return GEMMA_ERR_INVALID_ARG;
        const int st = check_paged(max_pages, page_size, n_pages);
        if (st != GEMMA_OK) return st;
        if ((long long)n_pages * n_kv > (1ll << 31) - 1) return GEMMA_ERR_UNSUPPORTED;
        c->pg = gemma::PagedLayout{block_table, max_pages, page_size, n_pages};
        c->cap = max_pages * page_size;
        return GEMMA_OK;
    }
    if (kv_capacity < 1) return GEMMA_ERR_INVALID_ARG;
    // key tiles start at multiples of 32 slots, a ring's at multiples of 128
    const int unit = kind == GEMMA_SLIDING_RING ? 128 : 32;
    if (kv_capacity % unit != 0 || kv_capacity > (1 << 30)) return GEMMA_ERR_UNSUPPORTED;
    c->cap = kv_capacity;
    c->ring = kind == GEMMA_SLIDING_RING ? kv_capacity : 0;
    return GEMMA_OK;
}

// The owner layer's pointers.
int q4_pointers(void* const* k_codes, void* const* k_scales, void* const* v_codes,
                void* const* v_scales, int owner, int k_eq_v, gemma::Q4Cache* c) {
    if (!k_codes || !k_scales || !k_codes[owner] || !k_scales[owner]) return GEMMA_ERR_INVALID_ARG;
    c->k_codes = static_cast<uint8_t*>(k_codes[owner]);
    c->k_scales = static_cast<__nv_bfloat16*>(k_scales[owner]);
    if (!aligned16(c->k_codes) || !aligned16(c->k_scales)) return GEMMA_ERR_INVALID_ARG;
    if (k_eq_v) return GEMMA_OK;
    if (!v_codes || !v_scales || !v_codes[owner] || !v_scales[owner]) return GEMMA_ERR_INVALID_ARG;
    c->v_codes = static_cast<uint8_t*>(v_codes[owner]);
    c->v_scales = static_cast<__nv_bfloat16*>(v_scales[owner]);
    if (!aligned16(c->v_codes) || !aligned16(c->v_scales)) return GEMMA_ERR_INVALID_ARG;
    return GEMMA_OK;
}

// One index unit is eight elements of one row; a sequence's units are counted in 32 bits.
bool q4_units_ok(long long rows, int n_kv, int head_dim) {
    return rows * n_kv <= (1ll << 30) / (head_dim / 8);
}

// Append (write_rows) or read-back of n rows per sequence.
int q4_rows(bool append, void* const* k_codes, void* const* k_scales, void* const* v_codes,
            void* const* v_scales, const int32_t* owner_map, int n_layers, int layer, void* k_rows,
            void* v_rows, const int32_t* pos, const int32_t* block_table, int max_pages,
            int page_size, int n_pages, int batch, int n, int kind, int n_kv, int head_dim,
            int kv_capacity, int k_eq_v, int dtype, uint32_t* device_error, void* stream) {
    if (batch < 0 || n < 0) return GEMMA_ERR_INVALID_ARG;
    if (dtype != GEMMA_BF16 && dtype != GEMMA_FP32) return GEMMA_ERR_INVALID_ARG;
    gemma::Q4Cache c;
    int st = q4_layout(kind, n_kv, head_dim, kv_capacity, block_table, max_pages, page_size,
                       n_pages, &c);
    if (st != GEMMA_OK) return st;
    int o = 0;
    st = resolve_owner(owner_map, n_layers, layer, &o);
    if (st != GEMMA_OK) return st;
    if (append && o != layer) return GEMMA_OK;  // a shared layer writes no cache
    if (n > c.cap) return GEMMA_ERR_CAPACITY;
    if (batch > 65535 || !q4_units_ok(n, n_kv, head_dim)) return GEMMA_ERR_UNSUPPORTED;
    if (batch == 0 || n == 0) return GEMMA_OK;
    st = q4_pointers(k_codes, k_scales, v_codes, v_scales, o, k_eq_v, &c);
    if (st != GEMMA_OK) return st;
    if (!k_rows || !pos || !aligned16(k_rows) || !aligned4(pos) || !aligned4(block_table) ||
        !aligned4(device_error))
        return GEMMA_ERR_INVALID_ARG;
    if (!k_eq_v && (!v_rows || !aligned16(v_rows))) return GEMMA_ERR_INVALID_ARG;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int f32 = dtype == GEMMA_FP32;
    const cudaError_t e =
        append ? gemma::launch_q4_append(c, k_rows, v_rows, pos, batch, n, head_dim, f32,
                                         device_error, n_sm, s)
               : gemma::launch_q4_read(c, k_rows, v_rows, pos, batch, n, head_dim, f32,
                                       device_error, n_sm, s);
    return e == cudaSuccess ? GEMMA_OK : GEMMA_ERR_CUDA;
}

// A step of at most this many rows (token, query head) per KV head attends straight over the
// 4-bit cache, which it unpacks once per 16 rows; a longer one over a dequantised copy, on the bf16
// kernels. Both sides in us (direct, copy), at this many rows and twice that, d = head_dim:
//   d 64, 16 / 1 heads, 16 x 1000 keys:  15.9, 20.0 and 24.9, 19.7
//   d 128, 8 / 2, 16 x 4096:             68.8, 76.0 and 121.6, 77.2
//   d 256, 16 / 8, 4 x window 1024:      31.9, 32.5 and 47.8, 31.9
//   d 512, 16 / 1, 4 x 4096:             42.1, 92.1 and 63, 77
// (at d 512 the copy's kernels have few CTAs for so few rows: one sequence of 16,384 keys takes
// 49 us at 256 rows against 268, 16 sequences of 8192 278 against 172).
constexpr long long q4_direct_rows(int head_dim) {
    return head_dim == 512 ? 192 : head_dim == 128 ? 128 : 64;
}

// CTAs of a step straight over the cache: one or a cluster of them per unit (sequence, KV head, row
// tile), or as many as the GPU holds at once, each with an equal share of the key tiles.
struct Q4Plan {
    int ctas, balanced, cluster;
    size_t o_bytes, info_off, ws_bytes;
};
Q4Plan q4_plan(int batch, int kind, int window, int n_q, int n_kv, int head_dim, int max_seq_len,
               int n_tok, int n_sm) {
    const long long T = gemma::kQ4KeyTile;
    const long long rows = (long long)n_tok * (n_q / n_kv);
    const int tile = gemma::q4_row_tile((int)rows);
    const long long units = (long long)batch * n_kv * ((rows + tile - 1) / tile);
    long long reach = kind == GEMMA_GLOBAL ? max_seq_len : (long long)window + n_tok - 1;
    if (reach > max_seq_len) reach = max_seq_len;
    const long long tiles = (reach + 2 * T - 2) / T;  // the first may start before the range
    const long long typical = (reach + T - 1) / T;
    const long long slots = (long long)n_sm * gemma::kQ4CtasPerSm;
    Q4Plan pl{(int)units, 0, 1, 0, 0, 0};
    // Three ways, in us (8 rows, 16 at head_dim 512): one CTA per unit / the best cluster / equal
    // shares with a merge launch. A tile of a lone CTA takes 0.6, 0.9, 1.25, 2.6 at head_dim 64 to
    // 512, a cluster's merge about 2, equal shares 4 and the longer the more units.
    //   head_dim 64, 2 units:    4 tiles 6.1 / 7.0 / 8.3, 8 tiles 8.7 / 7.5 / 8.5, 32 tiles 23 / 9.6 / 8.9
    //   head_dim 256, 2 units:   2 tiles 6.3 / 7.2 / 8.9, 4 tiles 8.9 / 7.7 / 9.0, 16 tiles 24 / 9.8 /
    //                            9.1, 64 tiles 84 / 17.5 / 10.6
    //   head_dim 256, 32 units:  3 tiles 7.8 / 8.7 / 11.6, 8 tiles 14.0 / 10.3 / 12.0, 32 tiles 44 /
    //                            16.4 / 18.1
    //   head_dim 256, 128 units: 3 tiles 10.1 / 10.9 / 13.9, 8 tiles 19.2 / 15.1 / 18.3
    //   head_dim 256, 512 units: 8 tiles 40.9 / - / 42.5, 12 tiles 56.3 / - / 55.3
    //   head_dim 512, 1 unit:    2 tiles 10.7 / 11.9 / 11.8, 8 tiles 26.8 / 12.1 / 11.9, 64 tiles 175 /
    //                            30.2 / 14.0
    //   head_dim 512, 32 units:  3 tiles 14.1 / 15.2 / 17.1, 16 tiles 48.6 / 21.8 / 23.4
    //   head_dim 512, 64 units of 128 tiles at most: 335 / - / 85; 400 units, 8 tiles: 68.8 / - / 84.5
    // Thousands of units need no shares (3200 units: 283, 283).
    const long long tile_ns = head_dim == 512 ? 2600 : head_dim == 256 ? 1250 : head_dim * 7;
    int most = 1;
    while (most < gemma::kQ4MaxCluster && units * most * 2 <= slots) most *= 2;
    // (a whole cache's lengths differ: half of it on average)
    long long share = units * (typical + 1) / slots / (kind == GEMMA_GLOBAL ? 2 : 1);
    if (share < 1) share = 1;
    // (clusters of 8 double up on SMs where there are many of them: 16 units of 8 tiles 10.5 us
    // against 9.2 by 4 at head_dim 256, 16.9 against 15.0 at 512)
    if (most == 8 && units > 8 && units < 32 &&
        (head_dim == 512 || (typical + 3) / 4 <= share + 2600 / tile_ns))
        most = 4;
    const long long part = (typical + most - 1) / most;  // tiles of a cluster's CTA
    const long long few = (512 / head_dim + 2) * (units < 64 ? 1 : units <= slots ? 2 : 3);
    const bool whole = typical <= few || units >= 16 * slots;
    if ((typical - part) * tile_ns >= (units < 32 ? 3000 : 3600) &&
        (whole || part <= share + 2600 / tile_ns)) {
        while ((typical + pl.cluster - 1) / pl.cluster > part) pl.cluster *= 2;
        pl.ctas = (int)units * pl.cluster;
        return pl;
    }
    if (whole) return pl;
    // (a balanced launch counts its tiles in 32 bits per KV head and row tile)
    if (batch > 4096 || batch * tiles > (1ll << 30)) return pl;
    pl.balanced = 1;
    long long c = units * (tiles + 1) < slots ? units * (tiles + 1) : slots;
    if (c > gemma::kQ4MaxShares) c = gemma::kQ4MaxShares;
    pl.ctas = (int)c;
    const size_t parts = (size_t)c * 2 * tile;
    pl.o_bytes = parts * head_dim * sizeof(float);
    pl.info_off = pl.o_bytes + (size_t)round_up((long long)(parts * 2 * sizeof(float)), 256);
    pl.ws_bytes = pl.info_off + (size_t)units * 8;
    return pl;
}

// Positions that a step of n_new queries can reach, at most: the slots of a dequantised copy.
int q4_expand_slots(int kind, int window, int max_seq_len, int n_new) {
    const long long reach = kind == GEMMA_GLOBAL ? max_seq_len : (long long)window + n_new - 1;
    return (int)(reach < max_seq_len ? reach : max_seq_len);
}

// Scratch of the attention over a dequantised copy: lengths, K rows, V rows, split partials.
struct Q4Expand {
    int slots;
    size_t k_off, v_off, plan_off, bytes;
};
Q4Expand q4_expand_plan(int batch, int kind, int window, int n_q, int n_kv, int head_dim,
                        int max_seq_len, int n_new, int k_eq_v, int n_sm) {
    Q4Expand e{};
    e.slots = q4_expand_slots(kind, window, max_seq_len, n_new);
    const size_t rows = (size_t)batch * n_kv * e.slots * head_dim * 2;
    e.k_off = (size_t)round_up(4ll * batch, 256);
    e.v_off = e.k_off + (size_t)round_up((long long)rows, 256);
    e.plan_off = e.v_off + (k_eq_v ? 0 : (size_t)round_up((long long)rows, 256));
    e.bytes = e.plan_off + make_plan(batch, kind == GEMMA_GLOBAL ? GEMMA_GLOBAL : GEMMA_SLIDING,
                                     window, n_q, n_kv, head_dim, e.slots, n_new, n_sm)
                               .ws_bytes;
    return e;
}

}  // namespace

int gemma_kv_append_q4(void* const* k_codes, void* const* k_scales, void* const* v_codes,
                       void* const* v_scales, const int32_t* owner_map, int n_layers, int layer,
                       const void* k_new, const void* v_new, const int32_t* write_pos,
                       const int32_t* block_table, int max_pages, int page_size, int n_pages,
                       int batch, int n_new, gemma_layer_kind kind, int n_kv, int head_dim,
                       int kv_capacity, int k_eq_v, gemma_dtype dtype, uint32_t* device_error,
                       void* stream) {
    return q4_rows(true, k_codes, k_scales, v_codes, v_scales, owner_map, n_layers, layer,
                   const_cast<void*>(k_new), const_cast<void*>(v_new), write_pos, block_table,
                   max_pages, page_size, n_pages, batch, n_new, kind, n_kv, head_dim, kv_capacity,
                   k_eq_v, dtype, device_error, stream);
}

int gemma_kv_read_q4(const void* const* k_codes, const void* const* k_scales,
                     const void* const* v_codes, const void* const* v_scales,
                     const int32_t* owner_map, int n_layers, int layer, void* k_out, void* v_out,
                     const int32_t* read_pos, const int32_t* block_table, int max_pages,
                     int page_size, int n_pages, int batch, int n_rows, gemma_layer_kind kind,
                     int n_kv, int head_dim, int kv_capacity, int k_eq_v, gemma_dtype dtype,
                     uint32_t* device_error, void* stream) {
    return q4_rows(false, const_cast<void* const*>(k_codes), const_cast<void* const*>(k_scales),
                   const_cast<void* const*>(v_codes), const_cast<void* const*>(v_scales),
                   owner_map, n_layers, layer, k_out, v_out, read_pos, block_table, max_pages,
                   page_size, n_pages, batch, n_rows, kind, n_kv, head_dim, kv_capacity, k_eq_v,
                   dtype, device_error, stream);
}

size_t gemma_attn_workspace_size_q4(int batch, gemma_layer_kind kind, int window, int n_q,
                                    int n_kv, int head_dim, int max_seq_len, int n_new,
                                    int k_eq_v) {
    if (batch < 0 || n_new < 1 || max_seq_len < n_new) return (size_t)-1;
    if (check_shape(kind, window, n_q, n_kv, head_dim, GEMMA_BF16) != GEMMA_OK) return (size_t)-1;
    // what the call refuses has no size
    const bool direct = (long long)n_new * (n_q / n_kv) <= q4_direct_rows(head_dim);
    if (batch > 65535 || n_kv > 32767 || max_seq_len > (1 << 30)) return (size_t)-1;
    if (!direct && !q4_units_ok(q4_expand_slots(kind, window, max_seq_len, n_new), n_kv, head_dim))
        return (size_t)-1;
    if (batch == 0) return 0;
    const int n_sm = sm_count();
    if (n_sm < 0) return (size_t)-1;
    if (direct)
        return q4_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_new, n_sm).ws_bytes;
    return q4_expand_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_new, k_eq_v,
                          n_sm)
        .bytes;
}

int gemma_attn_q4(void* out, const void* q, const void* const* k_codes,
                  const void* const* k_scales, const void* const* v_codes,
                  const void* const* v_scales, const int32_t* owner_map, int n_layers, int layer,
                  const int32_t* seq_lens, const int32_t* block_table, int max_pages,
                  int page_size, int n_pages, int max_seq_len, int n_new, int batch,
                  gemma_layer_kind kind, int window, int n_q, int n_kv, int head_dim, int k_eq_v,
                  int kv_capacity, float scale, float softcap, gemma_dtype dtype, void* workspace,
                  size_t workspace_bytes, uint32_t* device_error, void* stream) {
    if (n_new == 0 && batch >= 0) return GEMMA_OK;
    if (batch < 0 || n_new < 1) return GEMMA_ERR_INVALID_ARG;
    if (!std::isfinite(softcap) || softcap < 0.f) return GEMMA_ERR_INVALID_ARG;
    int st = check_shape(kind, window, n_q, n_kv, head_dim, dtype);
    if (st != GEMMA_OK) return st;
    if (dtype != GEMMA_BF16) return GEMMA_ERR_UNSUPPORTED;
    gemma::Q4Cache c;
    st = q4_layout(kind, n_kv, head_dim, kv_capacity, block_table, max_pages, page_size, n_pages,
                   &c);
    if (st != GEMMA_OK) return st;
    int o = 0;
    st = resolve_owner(owner_map, n_layers, layer, &o);
    if (st != GEMMA_OK) return st;
    if (max_seq_len < n_new || !std::isfinite(scale) || !(scale > 0.f))
        return GEMMA_ERR_INVALID_ARG;
    if (max_seq_len > (1 << 30)) return GEMMA_ERR_UNSUPPORTED;  // positions in 32 bits
    if (c.ring) {
        if ((long long)c.cap < (long long)window + n_new - 1) return GEMMA_ERR_CAPACITY;
    } else if (max_seq_len > c.cap) {
        return GEMMA_ERR_CAPACITY;
    }
    const bool direct = (long long)n_new * (n_q / n_kv) <= q4_direct_rows(head_dim);
    if (batch > 65535) return GEMMA_ERR_UNSUPPORTED;
    if (!direct && !q4_units_ok(q4_expand_slots(kind, window, max_seq_len, n_new), n_kv, head_dim))
        return GEMMA_ERR_UNSUPPORTED;
    if (batch == 0) return GEMMA_OK;
    st = q4_pointers(const_cast<void* const*>(k_codes), const_cast<void* const*>(k_scales),
                     const_cast<void* const*>(v_codes), const_cast<void* const*>(v_scales), o,
                     k_eq_v, &c);
    if (st != GEMMA_OK) return st;
    if (!out || !q || !seq_lens || !aligned16(out) || !aligned16(q) ||
        !aligned4(seq_lens) || !aligned4(block_table) || !aligned4(device_error))
        return GEMMA_ERR_INVALID_ARG;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (direct) {
        const Q4Plan pl =
            q4_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_new, n_sm);
        if (pl.ws_bytes > 0 &&
            (!workspace || workspace_bytes < pl.ws_bytes || !aligned16(workspace)))
            return GEMMA_ERR_WORKSPACE;
        RowsParams p{};
        p.q = q;
        p.k = c.k_codes;
        p.v = k_eq_v ? c.k_codes : c.v_codes;
        p.seq_lens = seq_lens;
        p.out = out;
        p.o_part = static_cast<float*>(workspace);
        p.ml_part = pl.ws_bytes ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                                           pl.o_bytes)
                                : nullptr;
        p.err = device_error;
        p.n_tok = n_new;
        p.n_q = n_q;
        p.n_kv = n_kv;
        p.G = n_q / n_kv;
        p.cap = c.cap;
        p.window = window;
        p.is_sliding = kind != GEMMA_GLOBAL;
        p.ring = c.ring;
        p.block_table = c.pg.block_table;
        p.page_size = c.pg.block_table ? c.pg.page_size : 0;
        p.max_pages = c.pg.max_pages;
        p.n_pages = c.pg.n_pages;
        p.k_eq_v = k_eq_v ? 1 : 0;
        p.max_seq_len = max_seq_len;
        p.scale_log2 = scale * 1.4426950408889634f;
        p.softcap = softcap;
        p.cap_inner = softcap > 0.f ? scale / softcap : 0.f;
        p.cap_log2 = softcap * 1.4426950408889634f;
        return gemma::launch_q4_attn(p, c, head_dim, batch, pl.ctas, pl.balanced, pl.cluster,
                                     static_cast<uint8_t*>(workspace) + pl.info_off, s) ==
                       cudaSuccess
                   ? GEMMA_OK
                   : GEMMA_ERR_CUDA;
    }
    const Q4Expand e = q4_expand_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len,
                                      n_new, k_eq_v, n_sm);
    if (!workspace || workspace_bytes < e.bytes || !aligned16(workspace))
        return GEMMA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int32_t* lens = reinterpret_cast<int32_t*>(ws);
    if (gemma::launch_q4_expand(c, ws + e.k_off, k_eq_v ? nullptr : ws + e.v_off, lens, seq_lens,
                                batch, n_new, max_seq_len, kind == GEMMA_GLOBAL ? 0 : window,
                                e.slots, head_dim, device_error, n_sm, s) != cudaSuccess)
        return GEMMA_ERR_CUDA;
    const void* kx = ws + e.k_off;
    const void* vx = ws + e.v_off;
    const int32_t self = 0;
    return attention(out, q, &kx, &vx, &self, 1, 0, lens, e.slots, n_new, batch,
                     kind == GEMMA_GLOBAL ? GEMMA_GLOBAL : GEMMA_SLIDING, window, n_q, n_kv,
                     head_dim, k_eq_v, e.slots, scale, softcap, GEMMA_BF16, ws + e.plan_off,
                     workspace_bytes - e.plan_off, device_error, stream);
}

int gemma_logit_sample(const void* logits, int batch, int vocab, gemma_dtype dtype, float softcap,
                       const float* temperature, const int32_t* top_k, const float* top_p,
                       const float* min_p, const float* uniform, int32_t* token_out,
                       void* workspace, size_t workspace_bytes, uint32_t* device_error,
                       void* stream) {
    if (batch < 0 || vocab < 1 || (dtype != GEMMA_BF16 && dtype != GEMMA_FP32))
        return GEMMA_ERR_INVALID_ARG;
    if (!std::isfinite(softcap) || softcap < 0.f) return GEMMA_ERR_INVALID_ARG;
    if (batch > 65535 || vocab > gemma::kSampleMaxVocab) return GEMMA_ERR_UNSUPPORTED;
    if (batch == 0) return GEMMA_OK;
    if (!logits || !uniform || !token_out || !aligned16(logits)) return GEMMA_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(temperature), static_cast<const void*>(top_k),
                          static_cast<const void*>(top_p), static_cast<const void*>(min_p),
                          static_cast<const void*>(uniform), static_cast<const void*>(token_out),
                          static_cast<const void*>(device_error)})
        if (!aligned4(x)) return GEMMA_ERR_INVALID_ARG;
    const size_t need = gemma::sample_workspace(batch, dtype == GEMMA_FP32);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return GEMMA_ERR_WORKSPACE;
    const gemma::SampleParams p{logits, temperature, top_k, top_p, min_p, uniform, token_out,
                                static_cast<int32_t*>(workspace),
                                reinterpret_cast<unsigned long long*>(
                                    static_cast<uint8_t*>(workspace) +
                                    gemma::sample_workspace(batch, 0)),
                                device_error, batch, vocab, softcap};
    const cudaError_t e =
        gemma::launch_sample(p, dtype == GEMMA_FP32, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMMA_OK : GEMMA_ERR_CUDA;
}

size_t gemma_logit_sample_workspace_size(int batch, int vocab, gemma_dtype dtype) {
    if (batch < 0 || batch > 65535 || vocab < 1 || vocab > gemma::kSampleMaxVocab ||
        (dtype != GEMMA_BF16 && dtype != GEMMA_FP32))
        return (size_t)-1;
    return gemma::sample_workspace(batch, dtype == GEMMA_FP32);
}

// ---------------------------------------------------------------------------------------------
// drafted trees
// ---------------------------------------------------------------------------------------------
namespace {

// How a bf16 step runs, by sizes alone.
enum { kTreeRows, kTreeTc, kTreePair };
struct TreePlan {
    int path;
    int n_split, chunk;    // kTreeRows: chunks of keys
    int deal;              // kTreeTc, kTreePair: how units are dealt out
    int workers, cluster;  // to CTAs or pairs; CTAs of a unit's cluster
    size_t o_bytes, ws_bytes;
};

// Key tiles of a step, at most; the unit that 32 bits have to count.
long long tree_tiles(int batch, int n_kv, long long rows, long long row_tile, long long reach,
                     long long keys) {
    return (long long)batch * n_kv * ((rows + row_tile - 1) / row_tile) * ((reach + keys - 1) / keys);
}
// Positions that a sequence's nodes can attend (rings and pages start at whole tiles).
long long tree_reach(int kind, int window, int max_seq_len, int n_nodes) {
    const long long reach = kind == GEMMA_GLOBAL ? max_seq_len : (long long)window - 1 + n_nodes;
    return (reach < max_seq_len ? reach : max_seq_len) + gemma::kTreeKeyTile - 1;
}

TreePlan tree_plan(int batch, int kind, int window, int n_q, int n_kv, int head_dim,
                   int max_seq_len, int n_nodes, int n_sm) {
    const long long T = gemma::kTreeKeyTile;
    const long long rows = (long long)n_nodes * (n_q / n_kv), units = (long long)batch * n_kv;
    const long long reach = tree_reach(kind, window, max_seq_len, n_nodes);
    TreePlan pl{};
    pl.n_split = 1;
    pl.chunk = 1 << 30;
    // Two SMs and 256 rows per tile, or one and 128. Head_dim 256 in us, pairs / single SMs: 61 nodes x 4
    // heads, 2 KV heads, 1 sequence of 8192 keys 20 / 20, 7 of 4800 35 / 37, 16 of 4096 46 / 60, 64 of 2048
    // (64 nodes) 75 / 112; with 128 rows or fewer a pair's second SM would have none.
    // Head_dim 512: pairs from 33 rows on, mma.sync before. 32 rows, 4 KV heads, 1024 keys, 1 sequence 14.1
    // on mma.sync, 13.8 on pairs, 32 sequences 53 and 88; 48 rows 21 and 14.3, 137 and 91.
    if (head_dim == 512 ? rows > gemma::kTreeRowsMax : head_dim == 256 && rows > 128) {
        const int halves = head_dim / 256;
        const long long u = units * ((rows + 255) / 256) * halves, nt = (reach + 127) / 128;
        const long long tiles = u * nt;
        pl.path = kTreePair;
        // A pair for each unit, without parts and their merge, where no unit has more than 8 (4) tiles above
        // an equal share (of one tile, or with all windows full): 8 x 1.4 us, 4 x 2.2. Equal shares / alone,
        // 14 units of 244 rows, head_dim 256: 2 tiles 11.2 / 9.1 us, 4 15.7 / 11.9, 8 21.2 / 17.7; 16 of 256,
        // head_dim 512, 4 tiles 17.3 / 13.9.
        const long long share = kind == GEMMA_GLOBAL ? 1 : (tiles + n_sm / 2 - 1) / (n_sm / 2);
        if (u <= n_sm / 2 && nt - share <= 8 / halves) {
            pl.workers = (int)u;
            pl.deal = gemma::kTreeAlone;
            return pl;
        }
        pl.workers = (int)(tiles < n_sm / 2 ? tiles : n_sm / 2);
        // Of more units than pairs whole ones to each, where they are that short: 184 units of 5 tiles, head_dim
        // 256, 56.6 / 45.1 us, 408 (of two halves) of 2, head_dim 512, 138 / 112.
        if (u > n_sm / 2 && nt <= 8 / halves) pl.deal = gemma::kTreeWhole;
        else pl.ws_bytes = gemma::tree_pair_workspace(batch, pl.workers);
        return pl;
    }
    // Up to 16 rows of head_dim 64 or 128 over many keys of not too few units: mma.sync takes a tile in less
    // time than one takes on tcgen05. 16 rows, tcgen05 / mma.sync, head_dim 64: 64 x 2 heads x 4096 keys 43 /
    // 30 us, 8 x 2 x 8192 20.9 / 15.5, 32 x 4 x 512 9.3 / 11.5, 1 x 4 x 32768 20.5 / 25.5; head_dim 128: 45.6 /
    // 50.1, 21.5 / 17.3, 10.2 / 12.7, 21.4 / 22.8.
    const bool few = head_dim <= 128 && rows <= 16 && units * reach >= 100000 && units >= 8 &&
                     (head_dim == 64 || units < 64);
    if (head_dim <= 256 && !few) {
        pl.path = kTreeTc;
        const long long keys = head_dim <= 128 ? 128 : 64;  // of a tile
        const long long tiles = tree_tiles(batch, n_kv, rows, 128, reach, keys);
        pl.workers = (int)(tiles < n_sm ? tiles : n_sm);
        pl.ws_bytes = gemma::tree_tc_workspace(head_dim, batch, pl.workers);
        // A cluster for each unit (no merge launch), where that ends no later than equal shares. In ns: a tile
        // takes 850 at head_dim 64 and 128 (of 128 keys) and 1012 at 256; the merge launch of equal shares
        // 4500 (TreeShare, which knows the lengths, counts what its parts take to write as well); a cluster's
        // exchange 1.0, 2.0 and 5.9 thousand with 32 rows of 256, 128 of 64, 128 of 256. One unit of 32 rows and
        // head_dim 256, clusters of 8 / shares: 1100 keys 9.6 / 10.2 us; 128 rows: 14.6 / 11.7; 128 units of 17
        // tiles, alone / shares: 30.6 / 34.4.
        const long long u = units * ((rows + 127) / 128);
        const long long nt = kind == GEMMA_SLIDING_RING ? (reach + keys - 1) / keys : (reach - T + keys) / keys;
        const long long tile_ns = head_dim == 256 ? 1012 : 850, merge_ns = 4500;
        const long long cluster_ns = 700 + (rows < 128 ? rows : 128) * head_dim * 16 / 100;
        long long best = (u * nt + n_sm - 1) / n_sm * tile_ns + merge_ns;
        for (int c = 1; c <= 8 && u * c <= n_sm; c *= 2) {
            const long long t = (nt + c - 1) / c * tile_ns + (c > 1 ? cluster_ns : 0);
            if (t <= best && (c == 1 || u <= gemma::tree_tc_clusters(head_dim, c))) {
                best = t;
                pl.cluster = c;
                pl.deal = gemma::kTreeAlone;
            }
        }
        // more units than SMs, all short: whole ones to each (equal shares / whole: 456 units of 6 tiles,
        // head_dim 64, 40 / 31 us)
        if (u > n_sm && nt * tile_ns <= 7500) pl.deal = gemma::kTreeWhole;
        if (pl.deal != gemma::kTreeShares) pl.ws_bytes = 0;
        return pl;
    }
    // chunks of keys: as many as keep one wave of CTAs, each of at least a tile
    long long n = (long long)n_sm * gemma::tree_ctas_per_sm(head_dim) / units;
    if (n > kMaxSplit) n = kMaxSplit;
    if (n < 1) n = 1;
    const long long chunk = round_up((reach + n - 1) / n, T);
    n = (reach + chunk - 1) / chunk;
    if (n <= 1) return pl;
    pl.n_split = (int)n;
    pl.chunk = (int)chunk;
    const size_t parts = (size_t)batch * n_q * n_nodes * n;
    pl.o_bytes = parts * head_dim * sizeof(float);
    pl.ws_bytes = pl.o_bytes + (size_t)round_up((long long)(parts * 2 * sizeof(float)), 256);
    return pl;
}

// Sizes that gemma_attn_tree refuses whatever the pointers.
int tree_sizes(int batch, int kind, int window, int n_q, int n_kv, int head_dim, int max_seq_len,
               int n_nodes, int dtype) {
    if (batch < 0 || n_nodes < 1 || max_seq_len < 1) return GEMMA_ERR_INVALID_ARG;
    const int st = check_shape(kind, window, n_q, n_kv, head_dim, dtype);
    if (st != GEMMA_OK) return st;
    if (n_nodes > gemma::kTreeMaxNodes || batch > 65535 || n_kv > 65535 || max_seq_len > (1 << 30))
        return GEMMA_ERR_UNSUPPORTED;
    // (one warp per row and slice of a merge, one CTA per row of the fp32 path)
    if ((long long)batch * n_q * n_nodes > (1ll << 30)) return GEMMA_ERR_UNSUPPORTED;
    // (key tiles are counted in 32 bits)
    if (tree_tiles(batch, n_kv, (long long)n_nodes * (n_q / n_kv), 128,
                   tree_reach(kind, window, max_seq_len, n_nodes), gemma::kTreeKeyTile) > (1ll << 30))
        return GEMMA_ERR_UNSUPPORTED;
    return GEMMA_OK;
}

}  // namespace

size_t gemma_attn_workspace_size_tree(int batch, gemma_layer_kind kind, int window, int n_q,
                                      int n_kv, int head_dim, int max_seq_len, int n_nodes) {
    if (tree_sizes(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_nodes, GEMMA_BF16) !=
        GEMMA_OK)
        return (size_t)-1;
    if (batch == 0) return 0;
    const int n_sm = sm_count();
    if (n_sm < 0) return (size_t)-1;
    return tree_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_nodes, n_sm).ws_bytes;
}

int gemma_attn_tree(void* out, const void* q, const void* const* k_cache,
                    const void* const* v_cache, const int32_t* owner_map, int n_layers, int layer,
                    const int32_t* seq_lens, const int32_t* parents, const int32_t* n_real,
                    const int32_t* block_table, int max_pages, int page_size, int n_pages,
                    int max_seq_len, int n_nodes, int batch, gemma_layer_kind kind, int window,
                    int n_q, int n_kv, int head_dim, int k_eq_v, int kv_capacity, float scale,
                    float softcap, gemma_dtype dtype, void* workspace, size_t workspace_bytes,
                    uint32_t* device_error, void* stream) {
    if (n_nodes == 0 && batch >= 0) return GEMMA_OK;
    if (!std::isfinite(softcap) || softcap < 0.f) return GEMMA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return GEMMA_ERR_INVALID_ARG;
    int st = tree_sizes(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_nodes, dtype);
    if (st != GEMMA_OK) return st;
    const bool ring = kind == GEMMA_SLIDING_RING;
    if (block_table) {
        if (ring) return GEMMA_ERR_INVALID_ARG;
        st = check_paged(max_pages, page_size, n_pages);
        if (st != GEMMA_OK) return st;
        if ((long long)n_pages * n_kv > (1ll << 31) - 1) return GEMMA_ERR_UNSUPPORTED;
        kv_capacity = max_pages * page_size;
    }
    if (kv_capacity < 1) return GEMMA_ERR_INVALID_ARG;
    if (kv_capacity > (1 << 30)) return GEMMA_ERR_UNSUPPORTED;
    if (ring) {
        if (kv_capacity % 128 != 0) return GEMMA_ERR_UNSUPPORTED;
        if ((long long)kv_capacity < (long long)window + n_nodes - 1) return GEMMA_ERR_CAPACITY;
    } else if (max_seq_len > kv_capacity) {
        return GEMMA_ERR_CAPACITY;
    }
    int o = 0;
    st = resolve_owner(owner_map, n_layers, layer, &o);
    if (st != GEMMA_OK) return st;
    if (batch == 0) return GEMMA_OK;
    if (!out || !q || !seq_lens || !parents || !k_cache || !k_cache[o]) return GEMMA_ERR_INVALID_ARG;
    if (!k_eq_v && (!v_cache || !v_cache[o])) return GEMMA_ERR_INVALID_ARG;
    const void* kc = k_cache[o];
    const void* vc = k_eq_v ? kc : v_cache[o];
    if (!aligned16(out) || !aligned16(q) || !aligned16(kc) || !aligned16(vc))
        return GEMMA_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(seq_lens), static_cast<const void*>(parents),
                          static_cast<const void*>(n_real), static_cast<const void*>(block_table),
                          static_cast<const void*>(device_error)})
        if (!aligned4(x)) return GEMMA_ERR_INVALID_ARG;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    const TreePlan pl =
        tree_plan(batch, kind, window, n_q, n_kv, head_dim, max_seq_len, n_nodes, n_sm);
    const bool bf16 = dtype == GEMMA_BF16;
    if (bf16 && pl.ws_bytes > 0 &&
        (!workspace || workspace_bytes < pl.ws_bytes || !aligned16(workspace)))
        return GEMMA_ERR_WORKSPACE;
    gemma::TreeParams tp{};
    RowsParams& p = tp.p;
    tp.parents = parents;
    tp.n_sm = n_sm;
    p.q = q;
    p.k = kc;
    p.v = vc;
    p.seq_lens = seq_lens;
    p.n_real = n_real;
    p.out = out;
    p.o_part = static_cast<float*>(workspace);
    p.ml_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.o_bytes);
    p.err = device_error;
    p.n_tok = n_nodes;
    p.n_q = n_q;
    p.n_kv = n_kv;
    p.G = n_q / n_kv;
    p.cap = kv_capacity;
    p.window = window;
    p.is_sliding = kind != GEMMA_GLOBAL;
    p.ring = ring ? kv_capacity : 0;
    p.block_table = block_table;
    p.page_size = block_table ? page_size : 0;
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.k_eq_v = k_eq_v ? 1 : 0;
    p.max_seq_len = max_seq_len;
    p.n_split = pl.n_split;
    p.chunk = pl.chunk;
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.softcap = softcap;
    // (finite, and so is 2 log2(e) times it: a score of zero stays one under the smallest cap)
    p.cap_inner = softcap > 0.f ? std::min(scale / softcap, FLT_MAX / 4) : 0.f;
    p.cap_log2 = softcap * 1.4426950408889634f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (!bf16) {
        e = gemma::launch_tree_f32(tp, head_dim, batch, s);
    } else if (pl.path == kTreeTc) {
        e = gemma::launch_tree_tc(tp, head_dim, batch, workspace, pl.workers, pl.cluster, pl.deal, s);
    } else if (pl.path == kTreePair) {
        e = gemma::launch_tree_pair(tp, head_dim, batch, workspace, pl.workers, pl.deal, s);
    } else {
        e = gemma::launch_tree_rows(tp, head_dim, batch, s);
        if (e == cudaSuccess && pl.n_split > 1) e = gemma::launch_tree_combine(tp, head_dim, batch, s);
    }
    return e == cudaSuccess ? GEMMA_OK : GEMMA_ERR_CUDA;
}

int gemma_tree_accept(const int32_t* tokens, const int32_t* parents, const int32_t* next,
                      const int32_t* n_real, const int32_t* seq_lens, int batch, int n_nodes,
                      int32_t* path_out, int32_t* n_keep_out, int32_t* token_out,
                      int32_t* lens_out, uint32_t* device_error, void* stream) {
    if (batch < 0 || n_nodes < 1) return GEMMA_ERR_INVALID_ARG;
    if (n_nodes > gemma::kTreeMaxNodes || batch > (1 << 24)) return GEMMA_ERR_UNSUPPORTED;
    if (batch == 0) return GEMMA_OK;
    if (!tokens || !parents || !next || !path_out || !n_keep_out || !token_out ||
        (lens_out && !seq_lens))
        return GEMMA_ERR_INVALID_ARG;
    for (const void* x :
         {static_cast<const void*>(tokens), static_cast<const void*>(parents),
          static_cast<const void*>(next), static_cast<const void*>(n_real),
          static_cast<const void*>(seq_lens), static_cast<const void*>(path_out),
          static_cast<const void*>(n_keep_out), static_cast<const void*>(token_out),
          static_cast<const void*>(lens_out), static_cast<const void*>(device_error)})
        if (!aligned4(x)) return GEMMA_ERR_INVALID_ARG;
    return gemma::launch_tree_accept(tokens, parents, next, n_real, seq_lens, batch, n_nodes,
                                     path_out, n_keep_out, token_out, lens_out, device_error,
                                     static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMMA_OK
               : GEMMA_ERR_CUDA;
}

int gemma_kv_keep(void* const* caches, int n_caches, const int32_t* write_pos, const int32_t* path,
                  const int32_t* n_keep, const int32_t* block_table, int max_pages, int page_size,
                  int n_pages, int batch, int n_nodes, gemma_layer_kind kind, int n_kv,
                  int kv_capacity, int row_bytes, uint32_t* device_error, void* stream) {
    if (batch < 0 || n_nodes < 1 || n_caches < 0 || n_kv < 1 || row_bytes < 2 || row_bytes % 2 != 0)
        return GEMMA_ERR_INVALID_ARG;
    if (kind != GEMMA_SLIDING && kind != GEMMA_GLOBAL && kind != GEMMA_SLIDING_RING)
        return GEMMA_ERR_INVALID_ARG;
    const bool ring = kind == GEMMA_SLIDING_RING;
    if (block_table) {
        if (ring) return GEMMA_ERR_INVALID_ARG;
        const int st = check_paged(max_pages, page_size, n_pages);
        if (st != GEMMA_OK) return st;
        kv_capacity = max_pages * page_size;
    }
    if (kv_capacity < 1) return GEMMA_ERR_INVALID_ARG;
    if (kv_capacity > (1 << 30) || n_nodes > gemma::kTreeMaxNodes || batch > 65535 ||
        (long long)n_kv * row_bytes > (1ll << 30))
        return GEMMA_ERR_UNSUPPORTED;
    if (ring && kv_capacity < n_nodes) return GEMMA_ERR_CAPACITY;
    if (batch == 0 || n_caches == 0) return GEMMA_OK;
    if (!caches || !write_pos || !path || !n_keep) return GEMMA_ERR_INVALID_ARG;
    for (int i = 0; i < n_caches; ++i)
        if (!caches[i] || !aligned16(caches[i])) return GEMMA_ERR_INVALID_ARG;
    // Rows move in place, each cache by threads of its own: none may share bytes with another.
    const uint64_t rows = block_table ? (uint64_t)n_pages * page_size : (uint64_t)batch * kv_capacity,
                   row = (uint64_t)n_kv * row_bytes;  // (below 2^61 and at most 2^30)
    const uint64_t size = rows > UINT64_MAX / row ? UINT64_MAX : rows * row;
    bool overlap = false;
    for (int i = 1; i < n_caches; ++i)
        for (int j = 0; j < i; ++j) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(caches[i]), b = reinterpret_cast<uintptr_t>(caches[j]);
            overlap |= (a > b ? a - b : b - a) < size;
        }
    if (overlap) return GEMMA_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(write_pos), static_cast<const void*>(path),
                          static_cast<const void*>(n_keep), static_cast<const void*>(block_table),
                          static_cast<const void*>(device_error)})
        if (!aligned4(x)) return GEMMA_ERR_INVALID_ARG;
    gemma::KeepLayout k{};
    k.write_pos = write_pos;
    k.path = path;
    k.n_keep = n_keep;
    k.pg = gemma::PagedLayout{block_table, max_pages, page_size, n_pages};
    k.n = n_nodes;
    k.n_kv = n_kv;
    k.cap = kv_capacity;
    k.ring = ring ? kv_capacity : 0;
    k.row_bytes = row_bytes;
    return gemma::launch_kv_keep(caches, n_caches, k, batch, device_error,
                                 static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMMA_OK
               : GEMMA_ERR_CUDA;
}

// ---------------------------------------------------------------------------------------------
// pages of a pool
// ---------------------------------------------------------------------------------------------
namespace {

int page_table(int32_t* block_table, int max_pages, int page_size, int n_pages, int32_t* page_refs,
               int batch, const uint32_t* device_error, gemma::PageTable* t) {
    if (batch < 0) return GEMMA_ERR_INVALID_ARG;
    const int st = check_paged(max_pages, page_size, n_pages);
    if (st != GEMMA_OK) return st;
    if (n_pages > gemma::kMaxPages || batch > 65535 ||
        (long long)batch * max_pages > (1ll << 31) - 1)
        return GEMMA_ERR_UNSUPPORTED;
    if (batch == 0) return GEMMA_OK;
    if (!block_table || !page_refs || !aligned4(block_table) || !aligned4(page_refs) ||
        !aligned4(device_error))
        return GEMMA_ERR_INVALID_ARG;
    *t = gemma::PageTable{block_table, page_refs, max_pages, page_size, n_pages, batch};
    return GEMMA_OK;
}

int page_pools(void* const* pools, const int32_t* pool_n_kv, const int32_t* pool_row_bytes,
               int n_pools, int page_size, int n_pages, const void* workspace,
               size_t workspace_bytes) {
    if (n_pools < 1 || !pools || !pool_n_kv || !pool_row_bytes) return GEMMA_ERR_INVALID_ARG;
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i] || !aligned16(pools[i]) || pool_n_kv[i] < 1 || pool_row_bytes[i] < 2 ||
            pool_row_bytes[i] % 2 != 0)
            return GEMMA_ERR_INVALID_ARG;
        // a page of up to 1 GB: the copies' units are counted in 32 bits
        if ((long long)pool_n_kv[i] * pool_row_bytes[i] > (1ll << 30) / page_size)
            return GEMMA_ERR_UNSUPPORTED;
    }
    if (!workspace || workspace_bytes < gemma::pages_workspace(n_pages) || !aligned16(workspace))
        return GEMMA_ERR_WORKSPACE;
    return GEMMA_OK;
}

}  // namespace

size_t gemma_pages_workspace_size(int n_pages) {
    if (n_pages < 1 || n_pages > gemma::kMaxPages) return (size_t)-1;
    return gemma::pages_workspace(n_pages);
}

int gemma_pages_free(int32_t* block_table, int max_pages, int page_size, int n_pages,
                     int32_t* page_refs, const int32_t* keep_from, const int32_t* keep_to,
                     int batch, uint32_t* device_error, void* stream) {
    gemma::PageTable t;
    const int st = page_table(block_table, max_pages, page_size, n_pages, page_refs, batch,
                              device_error, &t);
    if (st != GEMMA_OK || batch == 0) return st;
    if ((!keep_from && !keep_to) || !aligned4(keep_from) || !aligned4(keep_to))
        return GEMMA_ERR_INVALID_ARG;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    return gemma::launch_pages_free(t, keep_from, keep_to, device_error, n_sm,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMMA_OK
               : GEMMA_ERR_CUDA;
}

int gemma_pages_fork(int32_t* block_table, int max_pages, int page_size, int n_pages,
                     int32_t* page_refs, int32_t* seq_lens, const int32_t* src, const int32_t* dst,
                     int n, int batch, uint32_t* device_error, void* stream) {
    if (n < 0) return GEMMA_ERR_INVALID_ARG;
    gemma::PageTable t;
    const int st = page_table(block_table, max_pages, page_size, n_pages, page_refs, batch,
                              device_error, &t);
    if (st != GEMMA_OK || batch == 0 || n == 0) return st;
    if (n > batch) return GEMMA_ERR_INVALID_ARG;  // each fork needs a sequence of its own
    if (!seq_lens || !src || !dst || !aligned4(seq_lens) || !aligned4(src) || !aligned4(dst))
        return GEMMA_ERR_INVALID_ARG;
    return gemma::launch_pages_fork(t, seq_lens, src, dst, n, device_error,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMMA_OK
               : GEMMA_ERR_CUDA;
}

int gemma_pages_reserve(void* const* pools, const int32_t* pool_n_kv,
                        const int32_t* pool_row_bytes, int n_pools, int32_t* block_table,
                        int max_pages, int page_size, int n_pages, int32_t* page_refs,
                        const int32_t* seq_lens, const int32_t* n_add, int batch, void* workspace,
                        size_t workspace_bytes, uint32_t* device_error, void* stream) {
    gemma::PageTable t;
    int st = page_table(block_table, max_pages, page_size, n_pages, page_refs, batch, device_error,
                        &t);
    if (st != GEMMA_OK || batch == 0) return st;
    if (!seq_lens || !n_add || !aligned4(seq_lens) || !aligned4(n_add))
        return GEMMA_ERR_INVALID_ARG;
    st = page_pools(pools, pool_n_kv, pool_row_bytes, n_pools, page_size, n_pages, workspace,
                    workspace_bytes);
    if (st != GEMMA_OK) return st;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    return gemma::launch_pages_reserve(
               gemma::PagePools{pools, pool_n_kv, pool_row_bytes, n_pools}, t, seq_lens, n_add,
               workspace, device_error, n_sm, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMMA_OK
               : GEMMA_ERR_CUDA;
}

int gemma_pages_compact(void* const* pools, const int32_t* pool_n_kv,
                        const int32_t* pool_row_bytes, int n_pools, int32_t* block_table,
                        int max_pages, int page_size, int n_pages, int32_t* page_refs,
                        int32_t* n_used_out, int batch, void* workspace, size_t workspace_bytes,
                        uint32_t* device_error, void* stream) {
    gemma::PageTable t;
    int st = page_table(block_table, max_pages, page_size, n_pages, page_refs, batch, device_error,
                        &t);
    if (st != GEMMA_OK || batch == 0) return st;
    if (!aligned4(n_used_out)) return GEMMA_ERR_INVALID_ARG;
    st = page_pools(pools, pool_n_kv, pool_row_bytes, n_pools, page_size, n_pages, workspace,
                    workspace_bytes);
    if (st != GEMMA_OK) return st;
    const int n_sm = sm_count();
    if (n_sm < 0) return GEMMA_ERR_CUDA;
    return gemma::launch_pages_compact(
               gemma::PagePools{pools, pool_n_kv, pool_row_bytes, n_pools}, t, n_used_out,
               workspace, device_error, n_sm, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMMA_OK
               : GEMMA_ERR_CUDA;
}

}  // extern "C"
