// tree_tc.cu -- attention of a drafted tree with up to 128 rows per KV head and tile, on the
// 5th-generation tensor cores (tcgen05, one SM per tile). Definition in tree_attn.cu.
//
// A unit is one KV head of one sequence and 128 of its rows (nodes x G query heads). Per tile of 64 keys
// (128 at head_dim 64 and 128): S = Q K^T (M 128, N keys) into tensor memory, softmax by groups of four
// warps (a thread per row and 32 or 64 keys), P as bf16 back into tensor memory, O += P V (N = head_dim). A
// tile takes 1.05 us at head_dim 256 where its 64 KB are there in time; when all SMs load, memory gives 6.1
// TB/s or a tile in 1.6 us, so what is left to lose is the start, the end and the change from one unit to the
// next:
//  - the key tiles of all units form one sequence (lengths are known on the device alone), of which
//    every CTA takes an equal share; every warp works out the share by itself, from a scan of the
//    lengths, before the first barrier wait;
//  - barriers, tensor memory and tensor maps are set up before the wait for the previous kernel;
//  - S and P have two buffers each, so that S(t + 1) and P V(t - 1) run beside the softmax of t, and
//    loads run ahead, into the next unit too;
//  - a unit cut between CTAs leaves parts (O fp32 as it stands in tensor memory, four columns of all
//    rows after another, so that stores are of 512 consecutive bytes) for tree_merge_kernel; where there
//    are few units, a cluster shares a unit out and merges through distributed shared memory, and many
//    short ones are not cut.
// Measured: 16 trees of 32 over a ring of 1024 (128 units of 64 rows, head_dim 256) 30 us, 4.9 TB/s; one
// tree of 8 over a window of 512, 9 us.
// Warps: softmax and epilogue, then one that loads K and V, one that issues S, one that loads Q (the wait
// for the last S of the part before must not hold back the next part's keys) and one that issues P V (one
// thread issuing both lost 1000 of 2960 cycles per tile in its waits).
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "tc.cuh"
#include "tmap.h"
#include "tree.h"
#include "tree_dev.cuh"

namespace gemma {

namespace {

constexpr int kTcRows = 128;
constexpr int kTcMaxSlots = 12;
constexpr int kTcMaxCluster = 8;
constexpr int kTcBox = 64 * 128;  // 64 keys x 64 columns
constexpr int kTcQBox = kTcRows * 128;

template <int D, bool SOFTCAP>
struct TcLay {
    // Keys per tile: with 64 a tile takes 0.6 us whatever it holds, in the waits of its steps one after another
    // (152 units of 128 rows over 4096 keys, K as V, head_dim 64: 64 keys 46 us, 128 33; head_dim 128: 48 /
    // 36; one of 64 rows over 300 keys 6.5 / 7.2). At 256 O, S and P of 128 would not fit tensor memory.
    static constexpr int KEYS = D <= 128 ? 128 : 64, BOXES = KEYS / 64;
    // Groups of four softmax warps, 64 columns each or, where a soft-cap makes the softmax the bound, 32. One /
    // two at head_dim 256, 152 units of 4096 keys, no cap 97 us, a cap of 10 times the scores 102 / 98, of
    // twice 153 / 105.
    static constexpr int GROUPS = (D <= 128 ? 2 : 1) * (SOFTCAP ? 2 : 1);
    static constexpr int SOFT = 4 * GROUPS;                          // softmax warps
    static constexpr int THREADS = 32 * (SOFT + 4);
    static constexpr int COLS = KEYS / GROUPS;                       // a group's columns of S
    static constexpr int O_COLS = D / GROUPS < 32 ? 32 : D / GROUPS;    // and of O, where it has some
    static constexpr int O_GROUPS = D / O_COLS;
    static constexpr int SLOT = KEYS * D * 2, BLOCK = BOXES * kTcBox;  // a tile; 64 columns of it
    // Of a tile where memory does not hold it up, of one when all SMs load, and of parts and their merge: what
    // TreeShare weighs against each other.
    static constexpr int TILE_NS = D == 256 ? 1070 : 900, SHARE_NS = D == 256 ? 1630 : 900, MERGE_NS = 7500;
    // TMEM columns: O, S (two buffers), P (two buffers of packed bf16)
    static constexpr int O_COL = 0, S_COL = D, P_COL = S_COL + 2 * KEYS;
    static_assert(P_COL + KEYS <= 512, "tensor memory budget");
    static constexpr int EXTRA = 2 * (GROUPS > 1 ? GROUPS : 2) * 128 * 4 + 512;  // row maxima, barriers
    static constexpr int Q = kTcRows * D * 2;
    static constexpr int FIT = (232448 - Q - EXTRA) / SLOT;
    static constexpr int SLOTS = FIT > kTcMaxSlots ? kTcMaxSlots : FIT;
    static constexpr int Q_OFF = SLOTS * SLOT;
    static constexpr int MX_OFF = Q_OFF + Q;                         // row maxima [2][groups][128]
    static constexpr int BAR_OFF = MX_OFF + EXTRA - 512;
    static constexpr int SMEM = BAR_OFF + 512;
    static_assert(SMEM <= 232448 && (2 * kTcMaxSlots + 13) * 8 + 4 <= 512, "shared memory budget");
    // (a cluster's exchange lies in the ring)
    static_assert(SLOTS * SLOT >= kTcRows * D * 4, "shared memory budget");
    // CTAs of two clusters that waited for each other's tensor memory would wait for ever
    static_assert(2 * (SMEM + 1024) > 228 * 1024, "one CTA per SM");
};

GEMMA_DEVINL float2 ld_cluster_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
GEMMA_DEVINL void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c),
                 "f"(d)
                 : "memory");
}

}  // namespace

// Alone: a unit to each cluster of tp.workers CTAs, which share out its key tiles and merge their
// O through distributed shared memory (or, one CTA, write it): no second launch, no workspace
template <int D, bool SOFTCAP, int DEAL>
__global__ void __launch_bounds__(TcLay<D, SOFTCAP>::THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap qmap, const MergeParams tp) {
    using Lay = TcLay<D, SOFTCAP>;
    constexpr bool CLUSTER = DEAL == kTreeAlone;
    constexpr int KEYS = Lay::KEYS, BOXES = Lay::BOXES, kTcO = Lay::O_COL, kTcS = Lay::S_COL, kTcP = Lay::P_COL;
    constexpr int S = Lay::SLOTS, GROUPS = Lay::GROUPS, SOFT = Lay::SOFT, COLS = Lay::COLS;
    constexpr int O_COLS = Lay::O_COLS, O_GROUPS = Lay::O_GROUPS;
    pdl_launch_dependents();
    const RowsParams& p = tp.tp.p;
    extern __shared__ __align__(1024) uint8_t tc_smem[];
    uint8_t* smem = tc_smem;
    uint8_t* ring = smem;
    uint8_t* sQ = smem + Lay::Q_OFF;  // [D / 64][128][64] bf16
    float* mxs = reinterpret_cast<float*>(smem + Lay::MX_OFF);  // [2][groups][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
    uint64_t* empty = full + kTcMaxSlots;   // the MMAs that read the slot have completed
    uint64_t* q_full = empty + kTcMaxSlots;
    uint64_t* q_free = q_full + 1;          // a part's last S has completed
    uint64_t* s_full = q_full + 2;          // [2] S is in TMEM
    uint64_t* s_free = q_full + 4;          // [2] the softmax warps have read it
    uint64_t* p_full = q_full + 6;          // [2] P is in TMEM
    uint64_t* pv_done = q_full + 8;         // [2] P V has completed
    uint64_t* o_full = q_full + 10;         // a part's last P V has completed
    uint64_t* o_free = q_full + 11;         // O has been read
    uint32_t* tslot = reinterpret_cast<uint32_t*>(q_full + 12);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nops = p.k_eq_v ? 1 : 2;
    // Slots of K and of V of their own (K read as V: of both), so that an issuer sees every phase of the
    // barriers it waits on: a parity wait two phases behind passes at once.
    const int nk = nops == 2 ? (S + 1) / 2 : S, nv = S - nk;

    if (warp == SOFT) {
        if (lane == 0) {
            prefetch_map(&kmap);
            prefetch_map(&qmap);
            if (nops == 2) prefetch_map(&vmap);
            for (int s = 0; s < S; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&s_full[i], 1);
                mbar_init(&s_free[i], SOFT);
                mbar_init(&p_full[i], SOFT);
                mbar_init(&pv_done[i], 1);
            }
            mbar_init(q_full, 1);
            mbar_init(q_free, 1);
            mbar_init(o_full, 1);
            mbar_init(o_free, SOFT);
            fence_barrier_init();
        }
        __syncwarp();
    } else if (warp == SOFT + 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    pdl_wait();  // the previous kernel on the stream has completed
    const int n_cta = CLUSTER ? tp.workers : 1, cta = CLUSTER ? (int)cluster_rank() : 0;
    std::conditional_t<CLUSTER, TreeAlone<Lay::KEYS, kTcRows, 1>,
                       TreeShare<Lay::KEYS, kTcRows, 1, DEAL == kTreeWhole>> share;
    if constexpr (CLUSTER)
        share.init(tp, blockIdx.x / n_cta, cta, n_cta);
    else
        share.init(tp, blockIdx.x, blockIdx.x == 0 && warp == 0 && DEAL == kTreeShares, Lay::TILE_NS,
                   Lay::SHARE_NS, Lay::MERGE_NS);
    // softmax warps: the row's reference and sum (of the last part)
    float m = -INFINITY, l = 0.f;

    if (warp == SOFT) {
        // ------------------------------------ TMA producer --------------------------------------
        // K(0), V(0), K(1), ...
        TreeUnit U;
        bool ok = true;
        TreeRing rk, rv;
        while (share.next(tp, U)) {
            if (lane == 0) {
                for (int t = 0; t < U.n_tiles && ok; ++t) {
                    int row3[BOXES], slot0[BOXES];
#pragma unroll
                    for (int g = 0; g < BOXES; ++g) {
                        const int key = U.k_begin + t * KEYS + 64 * g;
                        if (g && p.page_size && key >= U.sq.len) {  // behind the last key: no page
                            row3[g] = p.n_pages * p.n_kv;
                            slot0[g] = 0;
                        } else if (!kv_place(p, U.b, U.kvh, key, row3[g], slot0[g])) {
                            report(p.err, GEMMA_DEVERR_PAGE);  // reads zeros
                            row3[g] = p.n_pages * p.n_kv;
                        }
                    }
                    for (int v = 0; v < nops && ok; ++v) {
                        TreeRing& ring_v = v ? rv : rk;
                        const int s = (v ? nk : 0) + ring_v.slot;
                        if (ring_v.use > 0) ok = mbar_wait(&empty[s], (ring_v.use - 1) & 1, p.err);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&full[s], Lay::SLOT);
#pragma unroll
                        for (int g = 0; g < BOXES; ++g)
#pragma unroll
                            for (int j = 0; j < D / 64; ++j)
                                tma_load_3d(ring + s * Lay::SLOT + j * Lay::BLOCK + g * kTcBox,
                                            v ? &vmap : &kmap, 64 * j, slot0[g], row3[g], &full[s]);
                        ring_v.step(v ? nv : nk);
                    }
                }
            }
            __syncwarp();
        }
        if (lane == 0) {
            // what was loaded has been read before the CTA may exit
            for (int s = 0; s < nk + nv && ok; ++s) {
                const int uses = s < nk ? rk.use + (s < rk.slot) : rv.use + (s - nk < rv.slot);
                if (uses > 0) ok = mbar_wait(&empty[s], (uses - 1) & 1, p.err);
            }
        }
        __syncwarp();
    } else if (warp == SOFT + 2) {
        // ------------------------------------- Q rows -------------------------------------------
        // a part's, once the last S of the part before has read the buffer
        TreeUnit U;
        bool ok = true;
        int ord = 0;
        for (; share.next(tp, U); ++ord) {
            if (ord > 0 && ok) ok = mbar_wait(q_free, (ord - 1) & 1, p.err);
            if (lane == 0 && ok) {
                mbar_arrive_expect_tx(q_full, Lay::Q);
#pragma unroll
                for (int j = 0; j < D / 64; ++j)  // (tokens past the bucket read 0)
                    tma_load_4d(sQ + j * kTcQBox, &qmap, 64 * j, U.kvh * p.G, U.rt * kTcRows / p.G,
                                U.b, q_full);
            }
            __syncwarp();
        }
        if constexpr (DEAL == kTreeWhole) tree_dead_rows<D, kTcRows>(tp, blockIdx.x, gridDim.x);
        if (ord > 0 && ok) mbar_wait(q_free, (ord - 1) & 1, p.err);  // (landed before the CTA exits)
    } else if (warp == SOFT + 1 || warp == SOFT + 3) {
        // ------------------------------ MMA issuers: S and P V ----------------------------------
        // An MMA is accepted only when the one before it is nearly done, so what an issuer spends
        // in waits is lost to the tensor core unless another one issues meanwhile.
        const bool is_s = warp == SOFT + 1;
        const uint32_t id_s = idesc_bf16(128, KEYS, 0, 0), id_pv = idesc_bf16(128, D, 0, 1);
        const uint64_t qd = smem_desc_sw128(smem_u32(sQ), 0, 1024);
        bool ok = true;
        TreeUnit U;
        int T = 0;  // tile of the share
        TreeRing rg;  // of K or of V
        const int n_slots = is_s || nops == 1 ? nk : nv, slot0 = is_s || nops == 1 ? 0 : nk;
        for (int ord = 0; share.next(tp, U); ++ord) {
            for (int t = 0; t < U.n_tiles; ++t, ++T, rg.step(n_slots)) {
                const bool last = t == U.n_tiles - 1;
                const int s = slot0 + rg.slot, buf = T & 1;
                uint8_t* tile = ring + s * Lay::SLOT;
                if (is_s) {
                    if (t == 0 && ok) ok = mbar_wait(q_full, ord & 1, p.err);
                    if (T >= 2 && ok) ok = mbar_wait(&s_free[buf], ((T >> 1) - 1) & 1, p.err);
                    if (ok) ok = mbar_wait(&full[s], rg.use & 1, p.err);
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t kd = smem_desc_sw128(smem_u32(tile), 0, 1024);
#pragma unroll
                        for (int j = 0; j < D / 64; ++j)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                umma_ss(tmem + kTcS + KEYS * buf,
                                        qd + (uint64_t)((j * kTcQBox + ks * 32) >> 4),
                                        kd + (uint64_t)((j * Lay::BLOCK + ks * 32) >> 4), id_s,
                                        (j | ks) ? 1u : 0u);
                        umma_commit(&s_full[buf]);
                        if (nops == 2) umma_commit(&empty[s]);
                        if (last) umma_commit(q_free);
                    }
                } else {
                    const int key0 = U.k_begin + t * KEYS, n_valid = U.sq.len - key0,
                              n_head = U.first - key0;
                    if (ok) ok = mbar_wait(&full[s], rg.use & 1, p.err);
                    if (n_valid < KEYS || n_head > 0) {
                        // rows outside of the sequence's keys may hold anything: zeros
                        for (int i = lane; i < KEYS * (D / 8); i += 32) {
                            const int key = i / (D / 8), ch = i - key * (D / 8);
                            if (key >= n_valid || key < n_head)
                                *reinterpret_cast<uint4*>(tile + (ch >> 3) * Lay::BLOCK + key * 128 +
                                                          (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (t == 0 && ord > 0 && ok) ok = mbar_wait(o_free, (ord - 1) & 1, p.err);
                    if (ok) ok = mbar_wait(&p_full[buf], (T >> 1) & 1, p.err);
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t vd = smem_desc_sw128(smem_u32(tile), Lay::BLOCK, 1024);
#pragma unroll
                        for (int kk = 0; kk < KEYS / 16; ++kk)
                            umma_ts(tmem + kTcO, tmem + kTcP + KEYS / 2 * buf + 8 * kk,
                                    vd + (uint64_t)((kk * 2048) >> 4), id_pv,
                                    (t == 0 && kk == 0) ? 0u : 1u);
                        umma_commit(&pv_done[buf]);
                        umma_commit(&empty[s]);
                        if (last) umma_commit(o_full);
                    }
                }
                __syncwarp();
            }
        }
    } else {
        // -------------------------------- softmax and epilogue ----------------------------------
        const int w = GROUPS == 1 ? 0 : warp >> 2, r = threadIdx.x & 127;  // group; row of the tile = TMEM lane
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tO = tmem + kTcO + O_COLS * w + lanes;
        bool ok = true;
        TreeUnit U;
        int T = 0, ord = 0, in_b = -1, in_rt = -1;  // T: tile of the share
        TreeRow row;
        for (; share.next(tp, U); ++ord) {
            const int base = U.sq.base, R = U.rt * kTcRows + r;
            if (U.b != in_b || U.rt != in_rt) {  // (the same for the next KV head of the sequence)
                in_b = U.b;
                in_rt = U.rt;
                row.find(tp.tp, U, R, threadIdx.x == 0);
            }
            const bool idle = __all_sync(0xffffffffu, row.lo == INT_MAX);  // no row of the warp attends
            m = -INFINITY;
            l = 0.f;
            for (int t = 0; t < U.n_tiles; ++t, ++T) {
                const int buf = T & 1;
                if (ok) ok = mbar_wait(&s_full[buf], (T >> 1) & 1, p.err);
                tc_fence_after();
                if (idle) {  // P = 0 (both buffers keep it for the rest of the part)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[buf]);
                    // (not before the other warps have arrived for P(T - 2))
                    if (T >= 2 && ok) ok = mbar_wait(&pv_done[buf], ((T >> 1) - 1) & 1, p.err);
                    if (t < 2) {
                        tc_fence_after();
                        uint32_t z[COLS / 2];
#pragma unroll
                        for (int e = 0; e < COLS / 2; ++e) z[e] = 0u;
                        tmem_store(tmem + kTcP + KEYS / 2 * buf + COLS / 2 * w + lanes, z);
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(&p_full[buf]);
                    continue;
                }
                float s[COLS];
                {
                    uint32_t v[COLS / 32][32];
#pragma unroll
                    for (int i = 0; i < COLS / 32; ++i)
                        tmem_ld32(tmem + kTcS + KEYS * buf + COLS * w + 32 * i + lanes, v[i]);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < COLS; ++e) s[e] = __uint_as_float(v[e / 32][e % 32]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[buf]);  // S(T + 2) may overwrite it
                float sl2 = p.scale_log2;  // scale > 0: the raw maximum scales to the maximum
                const int kt0 = U.k_begin + t * KEYS + COLS * w;
                if constexpr (SOFTCAP) {
                    tree_mask(s, row, kt0, base, 0.f);  // (they may be NaN)
                    tree_cap(s, p);
                    sl2 = 1.f;
                }
                tree_mask(s, row, kt0, base, -INFINITY);
                float mx = tree_max(s) * sl2;
                if constexpr (GROUPS > 1) {  // the row's maximum over the groups
                    float* mxb = mxs + buf * (128 * GROUPS);
                    mxb[w * 128 + r] = mx;
                    named_bar_sync(1 + (warp & 3), 32 * GROUPS);
#pragma unroll
                    for (int i = 0; i < GROUPS; ++i) mx = fmaxf(mx, mxb[i * 128 + r]);
                }
                const float m_prev = m;
                if (mx > m + kTrLazyLog2) {
                    l = m == -INFINITY ? 0.f : l * fast_exp2(m - mx);
                    m = mx;
                }
                // O rows whose reference moved: rescaled once P V(T - 1) has completed (a row
                // without keys so far has O = 0)
                const bool moved = t > 0 && m != m_prev && m_prev != -INFINITY;
                if (__any_sync(0xffffffffu, moved)) {
                    if (ok) ok = mbar_wait(&pv_done[buf ^ 1], ((T - 1) >> 1) & 1, p.err);
                    tc_fence_after();
                    const float alpha = moved ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll 1
                    for (int j = 0; j < (w < O_GROUPS ? O_COLS / 32 : 0); ++j) {
                        uint32_t v[32];
                        tmem_ld32(tO + j * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                        tmem_st32(tO + j * 32, v);
                    }
                    tmem_st_wait();
                }
                uint32_t pw[COLS / 2];
                l += tree_exp(s, sl2, m == -INFINITY ? 0.f : -m, pw);
                // the buffer is free once P V(T - 2) has completed
                if (T >= 2 && ok) ok = mbar_wait(&pv_done[buf], ((T >> 1) - 1) & 1, p.err);
                tc_fence_after();
                tmem_store(tmem + kTcP + KEYS / 2 * buf + COLS / 2 * w + lanes, pw);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[buf]);
            }
            // ---- the part's results ----
            if constexpr (GROUPS > 1) {
                // the row's sum over the groups, in the place of the other parity's maxima, which have been
                // read by all
                float* lx = mxs + (T & 1) * (128 * GROUPS);
                lx[w * 128 + r] = l;
                named_bar_sync(1 + (warp & 3), 32 * GROUPS);
                l = 0.f;
#pragma unroll
                for (int i = 0; i < GROUPS; ++i) l += lx[i * 128 + r];
                named_bar_sync(1 + (warp & 3), 32 * GROUPS);  // (before the next tile's maxima)
            }
            if (ok) ok = mbar_wait(o_full, ord & 1, p.err);
            tc_fence_after();
            if (CLUSTER && n_cta > 1) continue;
            const int n_rows = min(kTcRows, p.n_tok * p.G - U.rt * kTcRows);
            const int tk = R / p.G;
            __nv_bfloat16* out =
                reinterpret_cast<__nv_bfloat16*>(p.out) +
                (((size_t)U.b * p.n_tok + tk) * p.n_q + U.kvh * p.G + (R - tk * p.G)) * (size_t)D + O_COLS * w;
            float4* part = reinterpret_cast<float4*>(tp.part_o) +
                           ((size_t)max(U.slot, 0) * (D / 4) + O_COLS / 4 * w) * kTcRows + r;
            if (U.slot >= 0 && w == 0) tp.part_ml[(size_t)U.slot * kTcRows + r] = make_float2(m, l);
            const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
            if (w >= O_GROUPS && lane == 0) mbar_arrive(o_free);  // (has no columns)
#pragma unroll 1
            for (int j = 0; j < (w < O_GROUPS ? O_COLS / 32 : 0); ++j) {
                uint32_t v[32];
                tmem_ld32(tO + j * 32, v);
                tmem_ld_wait();
                if (j == O_COLS / 32 - 1) {  // O has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_free);
                }
                if (U.slot >= 0) {
                    if (idle) continue;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        part[(size_t)(j * 8 + q) * kTcRows] = make_float4(
                            __uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                            __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
                } else if (r < n_rows) {
                    tree_store32(out + j * 32, v, l, wide);
                }
            }
        }
        // the last commits have arrived before the CTA may exit
        for (int x = max(0, T - 2); x < T && ok; ++x) ok = mbar_wait(&pv_done[x & 1], (x >> 1) & 1, p.err);
    }
    if constexpr (CLUSTER) {
        // The CTAs of the cluster tell each other their rows' (m, l); then each scales its O by 2^(m - M)
        // and sends every CTA its slice of the columns; then each adds up its slice. The buffers are the
        // ring and the Q rows, which nobody reads any more behind the first barrier.
        const TreeUnit& U = share.U;
        const int w = GROUPS == 1 ? 0 : warp >> 2, r = threadIdx.x & 127, R = U.rt * kTcRows + r;
        const int n_rows = min(kTcRows, p.n_tok * p.G - U.rt * kTcRows), tk = R / p.G;
        __nv_bfloat16* out =
            reinterpret_cast<__nv_bfloat16*>(p.out) +
            (((size_t)U.b * p.n_tok + tk) * p.n_q + U.kvh * p.G + (R - tk * p.G)) * (size_t)D;
        if (U.sq.bad && U.kvh == 0 && U.rt == 0 && cta == 0 && threadIdx.x == 0) report(p.err, U.sq.bad);
        if (n_cta == 1) {
            if (U.n_tiles == 0 && warp < 4 && r < n_rows)  // no nodes
                for (int j = 0; j < D / 8; ++j)
                    reinterpret_cast<uint4*>(out)[j] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            const int lg = 31 - __clz(D / n_cta), slice = 1 << lg;  // columns (powers of two)
            if (warp < 4) reinterpret_cast<float2*>(sQ)[r] = make_float2(m, l);
            tc_fence_before();
            cluster_sync();
            tc_fence_after();
            float L = 0.f;
            uint32_t have = 0;  // CTAs that had keys of this row
            if (warp < SOFT) {
                float M = -INFINITY;
                float2 ml[kTcMaxCluster];
#pragma unroll
                for (int k = 0; k < kTcMaxCluster; ++k)
                    ml[k] = k < n_cta ? ld_cluster_f32x2(map_to_peer(sQ + 8 * r, k))
                                      : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int k = 0; k < kTcMaxCluster; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
                for (int k = 0; k < kTcMaxCluster; ++k) {
                    if (ml[k].x == -INFINITY) {
                        L += ml[k].y;  // (0; NaN where every score was)
                        continue;
                    }
                    have |= 1u << k;
                    L = fmaf(fast_exp2(ml[k].x - M), ml[k].y, L);
                }
                if (__any_sync(0xffffffffu, have >> cta & 1)) {
                    const float a = m == -INFINITY ? 0.f : fast_exp2(m - M);
                    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
#pragma unroll 1
                    for (int j = w * (O_COLS / 32); j < min(D / 32, (w + 1) * (O_COLS / 32)); ++j) {
                        uint32_t v[32];
                        tmem_ld32(tmem + kTcO + lanes + j * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 8; ++q) {  // four columns: [source][slice / 4][row]
                            const int col = j * 32 + 4 * q, to = col >> lg, c4 = (col & (slice - 1)) >> 2;
                            st_cluster_f32x4(
                                map_to_peer(ring + ((size_t)(cta * (slice / 4) + c4) * kTcRows + r) * 16, to),
                                __uint_as_float(v[4 * q]) * a, __uint_as_float(v[4 * q + 1]) * a,
                                __uint_as_float(v[4 * q + 2]) * a, __uint_as_float(v[4 * q + 3]) * a);
                        }
                    }
                }
            }
            cluster_sync();
            if (warp < SOFT && r < n_rows) {
                const float inv = 1.f / L;
                for (int c8 = w; c8 < slice / 8; c8 += GROUPS) {
                    float a[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = 0.f;
#pragma unroll
                    for (int k = 0; k < kTcMaxCluster; ++k) {
                        if (!(have >> k & 1)) continue;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 x = *reinterpret_cast<const float4*>(
                                ring + ((size_t)(k * (slice / 4) + 2 * c8 + h) * kTcRows + r) * 16);
                            a[4 * h] += x.x;
                            a[4 * h + 1] += x.y;
                            a[4 * h + 2] += x.z;
                            a[4 * h + 3] += x.w;
                        }
                    }
                    // (no keys: zeros)
                    reinterpret_cast<uint4*>(out + cta * slice)[c8] =
                        L == 0.f ? make_uint4(0u, 0u, 0u, 0u)
                                 : make_uint4(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv),
                                              pack_bf16(a[4] * inv, a[5] * inv), pack_bf16(a[6] * inv, a[7] * inv));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == SOFT + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------------------------
namespace {

struct TcScratch {
    size_t ml_off, before_off, bytes;
};
TcScratch tc_scratch(int head_dim, int batch, int workers) {
    TcScratch s;
    const size_t rows = (size_t)2 * workers * kTcRows;
    s.ml_off = rows * head_dim * sizeof(float);
    s.before_off = s.ml_off + rows * sizeof(float2);
    s.bytes = s.before_off + ((size_t)batch + 8) / 4 * 16;
    return s;
}

template <int D, bool SOFTCAP>
cudaError_t launch_tc(const TreeParams& tree, int batch, void* workspace, int workers, int cluster,
                      int deal, cudaStream_t st) {
    using Lay = TcLay<D, SOFTCAP>;
    const RowsParams& p = tree.p;
    using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, MergeParams);
    const Kernel kernels[3] = {tree_tc_kernel<D, SOFTCAP, kTreeShares>, tree_tc_kernel<D, SOFTCAP, kTreeAlone>,
                               tree_tc_kernel<D, SOFTCAP, kTreeWhole>};
    static std::atomic<bool> configured[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
        for (Kernel k : kernels) {
            const cudaError_t e =
                cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
            if (e != cudaSuccess) return e;
        }
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_relaxed);
    }
    CUtensorMap km, vm, qm;
    // [rows][slots][D]: rows = sequences x KV heads (pages x KV heads for a paged pool)
    const uint64_t slots = (uint64_t)(p.page_size ? p.page_size : p.cap);
    const uint64_t rows = (uint64_t)(p.page_size ? p.n_pages : batch) * p.n_kv;
    const uint64_t dims[3] = {(uint64_t)D, slots, rows};
    const uint64_t strides[2] = {(uint64_t)D * 2, slots * D * 2};
    const uint32_t box[3] = {64, 64, 1};
    if (!encode_bf16_sw128(&km, p.k, 3, dims, strides, box)) return cudaErrorInvalidValue;
    if (!encode_bf16_sw128(&vm, p.v, 3, dims, strides, box)) return cudaErrorInvalidValue;
    // Q [B][n_tok][n_q][D]: G heads of one KV head's group x 128 / G tokens are a row tile
    const uint64_t qdims[4] = {(uint64_t)D, (uint64_t)p.n_q, (uint64_t)p.n_tok, (uint64_t)batch};
    const uint64_t qstrides[3] = {(uint64_t)D * 2, (uint64_t)p.n_q * D * 2,
                                  (uint64_t)p.n_tok * p.n_q * D * 2};
    const uint32_t qbox[4] = {64, (uint32_t)p.G, (uint32_t)(kTcRows / p.G), 1};
    if (!encode_bf16_sw128(&qm, p.q, 4, qdims, qstrides, qbox)) return cudaErrorInvalidValue;
    MergeParams tp{};
    tp.tp = tree;
    tp.batch = batch;
    tp.n_rt = (p.n_tok * p.G + kTcRows - 1) / kTcRows;
    tp.workers = deal == kTreeAlone ? cluster : workers;
    tp.keys = Lay::KEYS;
    const Kernel kernel = kernels[deal];
    if (deal == kTreeAlone) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(tp.n_rt * batch * p.n_kv * cluster));
        cfg.blockDim = dim3(Lay::THREADS);
        cfg.dynamicSmemBytes = Lay::SMEM;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)cluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kernel, km, vm, qm, tp);
    }
    const TcScratch ws = tc_scratch(D, batch, workers);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    if (deal == kTreeShares) {
        tp.part_o = reinterpret_cast<float*>(base);
        tp.part_ml = reinterpret_cast<float2*>(base + ws.ml_off);
        tp.before = reinterpret_cast<int32_t*>(base + ws.before_off);
    }
    const cudaError_t e =
        launch_pdl(kernel, dim3(workers), dim3(Lay::THREADS), Lay::SMEM, st, km, vm, qm, tp);
    return e == cudaSuccess && deal == kTreeShares ? launch_tree_merge(tp, D, kTcRows, st) : e;
}

}  // namespace

template <int D>
static int clusters_fit(int cluster) {
    static std::atomic<int> cache[64][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int i = cluster == 2 ? 1 : cluster == 4 ? 2 : 3;
    if (dev >= 0 && dev < 64) {
        const int n = cache[dev][i].load(std::memory_order_relaxed);
        if (n > 0) return n;
    }
    if (cudaFuncSetAttribute(tree_tc_kernel<D, false, kTreeAlone>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             TcLay<D, false>::SMEM) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster * 64);
    cfg.blockDim = dim3(TcLay<D, false>::THREADS);
    cfg.dynamicSmemBytes = TcLay<D, false>::SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, tree_tc_kernel<D, false, kTreeAlone>, &cfg) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) cache[dev][i].store(n, std::memory_order_relaxed);
    return n;
}

int tree_tc_clusters(int head_dim, int cluster) {
    switch (head_dim) {
        case 64: return clusters_fit<64>(cluster);
        case 128: return clusters_fit<128>(cluster);
        case 256: return clusters_fit<256>(cluster);
    }
    return 0;
}

size_t tree_tc_workspace(int head_dim, int batch, int workers) {
    return tc_scratch(head_dim, batch, workers).bytes;
}

cudaError_t launch_tree_tc(const TreeParams& tp, int head_dim, int batch, void* workspace,
                           int workers, int cluster, int deal, cudaStream_t st) {
    auto launch = [&](auto plain, auto capped) {
        return (tp.p.softcap > 0.f ? capped : plain)(tp, batch, workspace, workers, cluster, deal, st);
    };
    switch (head_dim) {
        case 64: return launch(launch_tc<64, false>, launch_tc<64, true>);
        case 128: return launch(launch_tc<128, false>, launch_tc<128, true>);
        case 256: return launch(launch_tc<256, false>, launch_tc<256, true>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gemma
