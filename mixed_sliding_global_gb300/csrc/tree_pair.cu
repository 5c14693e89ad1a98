// tree_pair.cu -- attention of a drafted tree with many rows per KV head, at head_dim 256 and 512, on
// CTA pairs (tcgen05 with cta_group::2). Definition in tree_attn.cu.
//
// A unit is one KV head of one sequence, 256 of its rows (nodes x G query heads) and 256 columns of
// the output. A cluster of two CTAs runs each MMA as one instruction of M = 256: CTA c owns rows 128 c
// .. 128 c + 127 (its Q rows in shared memory, its S, P and O in tensor memory), and each CTA holds half
// of every B operand. Per tile of 128 keys:
//   S = Q K^T   N = 128 keys: CTA c holds keys 64 c .. 64 c + 63 of K, 32 KB per 256 columns;
//   O += P V    N = 256 columns: CTA c holds columns 128 c .. 128 c + 127 of V, 32 KB.
// Head_dim 512 is two units, one per half of O's columns (128 rows of all of them would fill the tensor
// memory), and each computes S over all 512 columns: 48 MMAs per tile where 32 would do, but no exchange
// of partial scores between CTAs, which costs more than the 16 (scores stay fp32 throughout).
//  - S has two buffers, and P(t) takes the place of S(t) in its buffer, so that S(t + 1) runs beside
//    the softmax of t and S(t + 2) waits for P V(t) alone: the tensor core always has an MMA group
//    that it may start;
//  - units are cut into equal shares of the key tiles, parts merged by tree_merge_kernel (TreeShare); short
//    ones are not: a pair has one (TreeAlone) or several;
//  - parts leave O as it stands in tensor memory, four columns of all rows after another, so that
//    stores are of 512 consecutive bytes;
//  - barriers, tensor memory and tensor maps are set up before the wait for the previous kernel.
// Warps of each CTA: softmax (two groups of four, with a soft-cap four: group w has columns 64 w .. (32 w
// ..) of S and 128 w .. (64 w ..) of O, the groups swap row maxima through shared memory); then one that
// loads K and V, two that issue S and P V (even CTA) or forward their slots' arrivals to the even CTA, whose
// MMAs read both halves (odd CTA), and one that loads Q. Barriers that the issuers wait on live in the even
// CTA and count arrivals from both; their commits arrive in both CTAs.
#include <atomic>
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "tc.cuh"
#include "tmap.h"
#include "tree.h"
#include "tree_dev.cuh"

namespace gemma {

namespace {

constexpr int kTpRows = 256, kTpKeys = 128;
constexpr int kTpBox = 64 * 128;      // TMA box: 64 keys x 64 columns
constexpr int kTpSlot = 4 * kTpBox;   // K: 64 keys x 256 columns; V: 128 keys x 128 columns
constexpr int kTpQBox = 128 * 128;
constexpr int kTpO = 0, kTpS = 256;   // TMEM columns: O; S / P, two buffers of 128

template <int D, bool SOFTCAP>
struct TpLay {
    // Groups of four softmax warps. A tile with a soft-cap is bound by the softmax, and four have more of
    // it in flight; without, two end earlier. Two / four, 76 units of 4096 keys, head_dim 256: no cap 64 /
    // 68 us, a cap of 10 times the scores 77 / 75, of twice 191 / 125 (with a reciprocal per score; now
    // 99); 76 units of 256 keys 15.6 / 16.8.
    static constexpr int GROUPS = SOFTCAP ? 4 : 2;
    static constexpr int SOFT = 4 * GROUPS;                  // softmax warps
    static constexpr int THREADS = 32 * (SOFT + 4);
    static constexpr int COLS = 128 / GROUPS, O_COLS = 256 / GROUPS;  // a group's columns of S and O
    static constexpr int KB = D / 256;                       // K slots of a tile
    static constexpr int K_SLOTS = D == 512 ? 2 : 3, V_SLOTS = D == 512 ? 1 : 2;
    static constexpr int SLOTS = K_SLOTS + V_SLOTS;
    static constexpr int Q = 128 * D * 2;
    static constexpr int Q_OFF = SLOTS * kTpSlot;
    static constexpr int MX_OFF = Q_OFF + Q;                 // row maxima [3][128], sums [2][128]
    static constexpr int BAR_OFF = MX_OFF + 5 * 128 * 4;
    static constexpr int SMEM = BAR_OFF + 256;
    static_assert(SMEM <= 232448, "shared memory budget");
};

}  // namespace

// A float's bits as an integer of the same order, and back.
GEMMA_DEVINL int tp_ordered(int x) { return x ^ ((x >> 31) & 0x7fffffff); }

// Alone: a unit to each pair, which writes zeros itself where there is nothing: no merge, no workspace
template <int D, bool SOFTCAP, int DEAL>
__global__ void __launch_bounds__(TpLay<D, SOFTCAP>::THREADS, 1)
    tree_pair_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ CUtensorMap qmap, const MergeParams mp) {
    using Lay = TpLay<D, SOFTCAP>;
    constexpr bool ALONE = DEAL == kTreeAlone;
    using PairShare = std::conditional_t<ALONE, TreeAlone<kTpKeys, kTpRows, Lay::KB>,
                                         TreeShare<kTpKeys, kTpRows, Lay::KB, DEAL == kTreeWhole>>;
    constexpr int KB = Lay::KB, NK = Lay::K_SLOTS, NV = Lay::V_SLOTS;
    constexpr int GROUPS = Lay::GROUPS, SOFT = Lay::SOFT, COLS = Lay::COLS, O_COLS = Lay::O_COLS;
    pdl_launch_dependents();
    const RowsParams& p = mp.tp.p;
    extern __shared__ __align__(1024) uint8_t tp_smem[];
    uint8_t* smem = tp_smem;
    uint8_t* sQ = smem + Lay::Q_OFF;                                 // [D / 64][128][64] bf16
    int* mxs = reinterpret_cast<int*>(smem + Lay::MX_OFF);           // [3][128], ordered as the floats
    float* lxs = reinterpret_cast<float*>(mxs + 3 * 128);            // [2][128]
    // full: this CTA's half has landed; pfull (even CTA): the odd CTA's has (forwarded); empty: the
    // MMAs that read the slot have completed (in both CTAs)
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
    uint64_t* pfull = full + 5;
    uint64_t* empty = full + 10;
    uint64_t* q_full = full + 15;   // this CTA's Q rows of a part have landed
    uint64_t* q_pfull = full + 16;  // even CTA: the odd CTA's have
    uint64_t* q_free = full + 17;   // a part's last S has completed (both CTAs)
    uint64_t* s_full = full + 18;   // [2] S is in TMEM (both CTAs)
    uint64_t* p_full = full + 20;   // [2] even CTA: both CTAs' P is in TMEM
    uint64_t* pv_done = full + 22;  // [2] P V has completed (both CTAs)
    uint64_t* o_full = full + 24;   // a part's last P V has completed (both CTAs)
    uint64_t* o_free = full + 25;   // even CTA: both CTAs have read O
    uint32_t* tslot = reinterpret_cast<uint32_t*>(full + 26);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t c = cluster_rank();
    const int worker = blockIdx.x / 2;

    for (int i = threadIdx.x; i < 3 * 128; i += Lay::THREADS) mxs[i] = INT_MIN;
    if (threadIdx.x == 32 * SOFT) {
        prefetch_map(&kmap);
        prefetch_map(&qmap);
        prefetch_map(&vmap);
        for (int s = 0; s < Lay::SLOTS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&pfull[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_pfull, 1);
        mbar_init(q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 2 * SOFT);  // both CTAs' softmax warps
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(o_free, 2 * SOFT);
        fence_barrier_init();
    }
    __syncthreads();
    // both CTAs run and their barriers exist before the pair's allocation and any remote arrival
    cluster_sync();
    if (warp == SOFT + 1) {
        tmem_alloc_pair(tslot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    pdl_wait();  // the previous kernel on the stream has completed
    PairShare share;
    if constexpr (ALONE) {
        share.init(mp, worker, 0, 1);
    } else {
        // (compute bound: a tile takes as long alone as when every SM works, and the parts and their merge as
        // long as six of them, three at head_dim 512. Whole / cut: 30 units of 10 tiles, head_dim 256, 23.6 /
        // 25.6 us; 50 of 10, head_dim 512, 32.9 / 36.6; 20 of 5 19.2 / 21.1)
        share.init(mp, worker, blockIdx.x == 0 && warp == 0 && DEAL == kTreeShares, 1000 * KB, 1000 * KB, 6000);
    }
    TreeUnit U{};
    bool ok = true;

    // rows of a V tile outside of the sequence's keys may hold anything: zeros (whole warp)
    auto zero_v = [&](uint8_t* tile, int t) {
        const int key0 = U.k_begin + t * kTpKeys, n_valid = U.sq.len - key0, n_head = U.first - key0;
        if (n_valid >= kTpKeys && n_head <= 0) return;
        for (int i = lane; i < kTpKeys * 16; i += 32) {
            const int key = i >> 4, ch = i & 15;
            if (key >= n_valid || key < n_head)
                *reinterpret_cast<uint4*>(tile + (ch >> 3) * 2 * kTpBox + key * 128 + (ch & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
    };

    if (warp == SOFT) {
        // -------------------------------------- K and V -----------------------------------------
        // in the order of their use: K(0), K(1), V(0), K(2), V(1), ..., into the next part too
        TreeRing rk, rv;
        auto place = [&](const TreeUnit& X, int key, int& row3, int& slot0) {
            if (p.page_size && key >= X.sq.len) {  // behind the last key: no page of the sequence's
                row3 = p.n_pages * p.n_kv;
                slot0 = 0;
            } else if (!kv_place(p, X.b, X.kvh, key, row3, slot0)) {
                report(p.err, GEMMA_DEVERR_PAGE);  // reads zeros
                row3 = p.n_pages * p.n_kv;
            }
        };
        auto load_k = [&](const TreeUnit& X, int t) {
            int row3, slot0;
            place(X, X.k_begin + t * kTpKeys + 64 * (int)c, row3, slot0);
#pragma unroll
            for (int a = 0; a < KB; ++a) {
                const int s = rk.slot;
                if (rk.use > 0 && ok) ok = mbar_wait(&empty[s], (rk.use - 1) & 1, p.err);
                if (!ok) return;
                mbar_arrive_expect_tx(&full[s], kTpSlot);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tma_load_3d(smem + s * kTpSlot + j * kTpBox, &kmap, 256 * a + 64 * j, slot0, row3,
                                &full[s]);
                rk.step(NK);
            }
        };
        auto load_v = [&](const TreeUnit& X, int t) {
            const int s = NK + rv.slot;
            if (rv.use > 0 && ok) ok = mbar_wait(&empty[s], (rv.use - 1) & 1, p.err);
            if (!ok) return;
            mbar_arrive_expect_tx(&full[s], kTpSlot);
            // two blocks of 64 columns, each of 128 keys in two boxes
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                int row3, slot0;
                place(X, X.k_begin + t * kTpKeys + 64 * g, row3, slot0);
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
                    tma_load_3d(smem + s * kTpSlot + blk * 2 * kTpBox + g * kTpBox, &vmap,
                                256 * X.half + 128 * (int)c + 64 * blk, slot0, row3, &full[s]);
            }
            rv.step(NV);
        };
        TreeUnit prev;
        int prev_t = -1;
        while (share.next(mp, U)) {
            if (lane == 0) {
                for (int t = 0; t < U.n_tiles && ok; ++t) {
                    load_k(U, t);
                    if (prev_t >= 0) load_v(t ? U : prev, prev_t);
                    prev_t = t;
                }
                prev = U;
            }
            __syncwarp();
        }
        if (lane == 0) {
            if (prev_t >= 0) load_v(prev, prev_t);
            // what was loaded has been read before the CTA may exit
            for (int s = 0; s < NK + NV; ++s) {
                const int uses = s < NK ? rk.use + (s < rk.slot) : rv.use + (s - NK < rv.slot);
                if (uses > 0 && ok) ok = mbar_wait(&empty[s], (uses - 1) & 1, p.err);
            }
        }
        __syncwarp();
    } else if (warp == SOFT + 3) {
        // ---------------------------------------- Q ---------------------------------------------
        // a part's rows, once the last S of the part before has read the buffer
        int ord = 0;
        for (; share.next(mp, U); ++ord) {
            if (ord > 0 && ok) ok = mbar_wait(q_free, (ord - 1) & 1, p.err);
            if (lane == 0 && ok) {
                mbar_arrive_expect_tx(q_full, Lay::Q);
#pragma unroll
                for (int j = 0; j < D / 64; ++j)  // (tokens past the bucket read 0)
                    tma_load_4d(sQ + j * kTpQBox, &qmap, 64 * j, U.kvh * p.G,
                                (U.rt * kTpRows + 128 * (int)c) / p.G, U.b, q_full);
            }
            __syncwarp();
        }
        if constexpr (DEAL == kTreeWhole) tree_dead_rows<D, kTpRows>(mp, blockIdx.x, gridDim.x);
        if (ord > 0 && ok) mbar_wait(q_free, (ord - 1) & 1, p.err);  // (landed before the CTA exits)
    } else if (c == 0 && warp == SOFT + 1) {
        // ------------------------------------- S issuer -----------------------------------------
        const uint32_t id_s = idesc_bf16(256, kTpKeys, 0, 0);
        const uint64_t qd = smem_desc_sw128(smem_u32(sQ), 0, 1024);
        TreeRing rk;
        int T = 0;  // tile of the share
        for (int ord = 0; share.next(mp, U); ++ord) {
            for (int t = 0; t < U.n_tiles; ++t, ++T) {
                const int buf = T & 1;
                if (t == 0 && ok) {
                    ok = mbar_wait(q_full, ord & 1, p.err);
                    if (ok) ok = mbar_wait(q_pfull, ord & 1, p.err);
                }
                // P(T - 2) lies in the buffer until its P V has completed
                if (T >= 2 && ok) ok = mbar_wait(&pv_done[buf], ((T >> 1) - 1) & 1, p.err);
#pragma unroll
                for (int a = 0; a < KB; ++a) {
                    const int s = rk.slot;
                    if (ok) ok = mbar_wait(&full[s], rk.use & 1, p.err);
                    if (ok) ok = mbar_wait(&pfull[s], rk.use & 1, p.err);
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t kd = smem_desc_sw128(smem_u32(smem + s * kTpSlot), 0, 1024);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                umma_ss_pair(tmem + kTpS + 128 * buf,
                                             qd + (uint64_t)(((4 * a + j) * kTpQBox + ks * 32) >> 4),
                                             kd + (uint64_t)((j * kTpBox + ks * 32) >> 4), id_s,
                                             (a | j | ks) ? 1u : 0u);
                        umma_commit_pair(&empty[s], 3);
                        if (a == KB - 1) {
                            umma_commit_pair(&s_full[buf], 3);
                            if (t == U.n_tiles - 1) umma_commit_pair(q_free, 3);
                        }
                    }
                    __syncwarp();
                    rk.step(NK);
                }
            }
        }
    } else if (c == 0 && warp == SOFT + 2) {
        // ------------------------------------ P V issuer ----------------------------------------
        const uint32_t id_pv = idesc_bf16(256, 256, 0, 1);
        TreeRing rv;
        int T = 0;
        for (int ord = 0; share.next(mp, U); ++ord) {
            for (int t = 0; t < U.n_tiles; ++t, ++T, rv.step(NV)) {
                const int s = NK + rv.slot, buf = T & 1;
                uint8_t* tile = smem + s * kTpSlot;
                if (ok) ok = mbar_wait(&full[s], rv.use & 1, p.err);
                zero_v(tile, t);
                if (ok) ok = mbar_wait(&pfull[s], rv.use & 1, p.err);
                // a part's first P V overwrites O: the part before has been read
                if (t == 0 && ord > 0 && ok) ok = mbar_wait(o_free, (ord - 1) & 1, p.err);
                if (ok) ok = mbar_wait(&p_full[buf], (T >> 1) & 1, p.err);
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t vd = smem_desc_sw128(smem_u32(tile), 2 * kTpBox, 1024);
#pragma unroll
                    for (int kk = 0; kk < kTpKeys / 16; ++kk)
                        umma_ts_pair(tmem + kTpO, tmem + kTpS + 128 * buf + 8 * kk,
                                     vd + (uint64_t)((kk * 2048) >> 4), id_pv,
                                     (t == 0 && kk == 0) ? 0u : 1u);
                    umma_commit_pair(&pv_done[buf], 3);
                    umma_commit_pair(&empty[s], 3);
                    if (t == U.n_tiles - 1) umma_commit_pair(o_full, 3);
                }
                __syncwarp();
            }
        }
    } else if (c == 1 && warp == SOFT + 1) {
        // --------------------- odd CTA: arrivals of Q and K, to the even CTA --------------------
        const uint32_t pfull0 = map_to_peer(&pfull[0], 0), q_pfull0 = map_to_peer(q_pfull, 0);
        TreeRing rk;
        for (int ord = 0; share.next(mp, U); ++ord) {
            if (ok) ok = mbar_wait(q_full, ord & 1, p.err);
            if (lane == 0) mbar_arrive_remote(q_pfull0);
            __syncwarp();
            for (int t = 0; t < U.n_tiles * KB; ++t, rk.step(NK)) {
                if (ok) ok = mbar_wait(&full[rk.slot], rk.use & 1, p.err);
                if (lane == 0) mbar_arrive_remote(pfull0 + 8u * (uint32_t)rk.slot);
                __syncwarp();
            }
        }
    } else if (c == 1 && warp == SOFT + 2) {
        // ------------------------- odd CTA: arrivals of V, edges zeroed -------------------------
        const uint32_t pfull0 = map_to_peer(&pfull[0], 0);
        TreeRing rv;
        while (share.next(mp, U)) {
            for (int t = 0; t < U.n_tiles; ++t, rv.step(NV)) {
                const int s = NK + rv.slot;
                if (ok) ok = mbar_wait(&full[s], rv.use & 1, p.err);
                zero_v(smem + s * kTpSlot, t);
                if (lane == 0) mbar_arrive_remote(pfull0 + 8u * (uint32_t)s);
                __syncwarp();
            }
        }
    } else if (warp < SOFT) {
        // -------------------------------- softmax and epilogue ----------------------------------
        const int w = warp >> 2, r = threadIdx.x & 127;  // group; row of this CTA = TMEM lane
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tO = tmem + kTpO + O_COLS * w + lanes;
        const uint32_t p_full0 = map_to_peer(p_full, 0), o_free0 = map_to_peer(o_free, 0);
        int T = 0, ord = 0, in_b = -1, in_rt = -1, mx_at = 0;  // T: tile of the share
        TreeRow row;
        bool more = share.next(mp, U);
        for (; more; ++ord) {
            const int R = U.rt * kTpRows + 128 * (int)c + r;
            if (U.b != in_b || U.rt != in_rt) {  // (the same for the next half or KV head)
                in_b = U.b;
                in_rt = U.rt;
                row.find(mp.tp, U, R, c == 0 && threadIdx.x == 0);
            }
            float m = -INFINITY, l = 0.f;  // l: this group's columns
            for (int t = 0; t < U.n_tiles; ++t, ++T) {
                const int buf = T & 1;
                const uint32_t tSP = tmem + kTpS + 128 * buf + lanes;
                if (ok) ok = mbar_wait(&s_full[buf], (T >> 1) & 1, p.err);
                tc_fence_after();
                float s[COLS];
                {
                    uint32_t v[COLS / 32][32];
#pragma unroll
                    for (int i = 0; i < COLS / 32; ++i) tmem_ld32(tSP + COLS * w + 32 * i, v[i]);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < COLS; ++e) s[e] = __uint_as_float(v[e / 32][e % 32]);
                }
                tc_fence_before();  // (P takes the place of S behind the groups' barrier)
                float sl2 = p.scale_log2;  // scale > 0: the raw maximum scales to the maximum
                const int kt0 = U.k_begin + t * kTpKeys + COLS * w;
                if constexpr (SOFTCAP) {
                    tree_mask(s, row, kt0, U.sq.base, 0.f);  // (they may be NaN)
                    tree_cap(s, p);
                    sl2 = 1.f;
                }
                tree_mask(s, row, kt0, U.sq.base, -INFINITY);
                float mx = tree_max(s) * sl2;
                // the row's maximum over the groups (of two, an exchange: 2 us less of 178 for 16 trees of 512
                // rows over 16k keys than the atomics; of four, it would take 4 KB more than there are)
                if constexpr (GROUPS == 2) {
                    float* mxb = reinterpret_cast<float*>(mxs) + buf * 256;
                    mxb[w * 128 + r] = mx;
                    named_bar_sync(1, 32 * SOFT);
                    mx = fmaxf(mx, mxb[(w ^ 1) * 128 + r]);
                } else {
                    // three places in turn: the one that the tile after the next takes was read by all
                    // before this barrier
                    atomicMax(mxs + mx_at * 128 + r, tp_ordered(__float_as_int(mx)));
                    named_bar_sync(1, 32 * SOFT);
                    mx = __int_as_float(tp_ordered(mxs[mx_at * 128 + r]));
                    mx_at = mx_at == 2 ? 0 : mx_at + 1;
                    if (w == 0) mxs[(mx_at == 2 ? 0 : mx_at + 1) * 128 + r] = INT_MIN;
                }
                tc_fence_after();
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
                    for (int j = 0; j < O_COLS / 32; ++j) {
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
                tmem_store(tSP + COLS / 2 * w, pw);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(p_full0 + 8u * (uint32_t)buf);
            }

            // ---- the part's results ----
            const TreeUnit D0 = U;
            const TreeRow row0 = row;
            more = share.next(mp, U);
            if (ok) ok = mbar_wait(o_full, ord & 1, p.err);
            tc_fence_after();
            // the row's sum over the groups
            if constexpr (GROUPS == 2) {
                // (in the place of the other parity's maxima, which have been read by all)
                float* lx = reinterpret_cast<float*>(mxs) + (T & 1) * 256;
                lx[w * 128 + r] = l;
                named_bar_sync(2, 32 * SOFT);
                l += lx[(w ^ 1) * 128 + r];
                named_bar_sync(2, 32 * SOFT);  // (before the next tile's maxima)
            } else {
                if (w >= 2) lxs[(w - 2) * 128 + r] = l;
                named_bar_sync(2, 32 * SOFT);
                if (w < 2) l += lxs[w * 128 + r];
                if (w == 1) lxs[128 + r] = l;
                named_bar_sync(2, 32 * SOFT);
                if (w == 0) lxs[r] = l += lxs[128 + r];
                named_bar_sync(2, 32 * SOFT);
                l = lxs[r];
            }
            const int n_rows = p.n_tok * p.G - (D0.rt * kTpRows + 128 * (int)c);  // of this CTA
            const bool idle = __all_sync(0xffffffffu, row0.lo == INT_MAX);
            const int tk = R / p.G;
            __nv_bfloat16* out =
                reinterpret_cast<__nv_bfloat16*>(p.out) +
                (((size_t)D0.b * p.n_tok + tk) * p.n_q + D0.kvh * p.G + (R - tk * p.G)) * (size_t)D +
                256 * D0.half + O_COLS * w;
            const size_t piece = (size_t)max(D0.slot, 0) * 2 + c;
            float4* part = reinterpret_cast<float4*>(mp.part_o) + (piece * 64 + O_COLS / 4 * w) * 128 + r;
            if (D0.slot >= 0 && w == 0) mp.part_ml[piece * 128 + r] = make_float2(m, l);
            const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll 1
            for (int j = 0; j < O_COLS / 32; ++j) {
                uint32_t v[32];
                tmem_ld32(tO + j * 32, v);
                tmem_ld_wait();
                if (j == O_COLS / 32 - 1) {  // O has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(o_free0);
                }
                if (D0.slot >= 0) {
                    if (idle) continue;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        part[(size_t)(j * 8 + q) * 128] = make_float4(
                            __uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                            __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
                } else if (r < n_rows) {
                    tree_store32(out + j * 32, v, l, wide);
                }
            }
        }
        // the last commits have arrived before the CTA may exit
        for (int x = max(0, T - 2); x < T && ok; ++x)
            ok = mbar_wait(&pv_done[x & 1], (x >> 1) & 1, p.err);
    }
    if constexpr (ALONE) {
        const TreeUnit& X = share.U;
        const int r = threadIdx.x, n_rows = p.n_tok * p.G - (X.rt * kTpRows + 128 * (int)c);
        if (X.sq.bad && X.kvh == 0 && X.rt == 0 && X.half == 0 && c == 0 && r == 0) report(p.err, X.sq.bad);
        if (X.n_tiles == 0 && r < min(128, n_rows)) {  // no nodes
            const int R = X.rt * kTpRows + 128 * (int)c + r, tk = R / p.G;
            uint4* out = reinterpret_cast<uint4*>(
                reinterpret_cast<__nv_bfloat16*>(p.out) +
                (((size_t)X.b * p.n_tok + tk) * p.n_q + X.kvh * p.G + (R - tk * p.G)) * (size_t)D +
                256 * X.half);
            for (int j = 0; j < 32; ++j) out[j] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA arrives on another's barriers any more
    if (warp == SOFT + 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------------------------
namespace {

struct TpScratch {
    size_t ml_off, before_off, bytes;
};
TpScratch tp_scratch(int batch, int workers) {
    TpScratch s;
    const size_t rows = (size_t)2 * workers * kTpRows;
    s.ml_off = rows * 256 * sizeof(float);
    s.before_off = s.ml_off + rows * sizeof(float2);
    s.bytes = s.before_off + ((size_t)batch + 8) / 4 * 16;
    return s;
}

template <int D, bool SOFTCAP, int DEAL>
cudaError_t launch_tp(const TreeParams& tree, int batch, void* workspace, int workers, cudaStream_t st) {
    using Lay = TpLay<D, SOFTCAP>;
    const RowsParams& p = tree.p;
    auto kernel = tree_pair_kernel<D, SOFTCAP, DEAL>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(2 * workers);
    cfg.blockDim = dim3(Lay::THREADS);
    cfg.dynamicSmemBytes = Lay::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // per device: the shared-memory attribute, and how many clusters fit at once
    static std::atomic<int> clusters_fit[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    int fit = dev >= 0 && dev < 64 ? clusters_fit[dev].load(std::memory_order_relaxed) : 0;
    if (fit <= 0) {
        cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (fit < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 64) clusters_fit[dev].store(fit, std::memory_order_relaxed);
    }
    if (DEAL != kTreeAlone && workers > fit) workers = fit;
    cfg.gridDim = dim3(2 * workers);
    CUtensorMap km, vm, qm;
    // [rows][slots][D]: rows = sequences x KV heads (pages x KV heads for a paged pool)
    const uint64_t slots = (uint64_t)(p.page_size ? p.page_size : p.cap);
    const uint64_t rows = (uint64_t)(p.page_size ? p.n_pages : batch) * p.n_kv;
    const uint64_t dims[3] = {(uint64_t)D, slots, rows};
    const uint64_t strides[2] = {(uint64_t)D * 2, slots * D * 2};
    const uint32_t box[3] = {64, 64, 1};
    if (!encode_bf16_sw128(&km, p.k, 3, dims, strides, box)) return cudaErrorInvalidValue;
    if (!encode_bf16_sw128(&vm, p.v, 3, dims, strides, box)) return cudaErrorInvalidValue;
    // Q [B][n_tok][n_q][D]: G heads of one KV head's group x 128 / G tokens are a CTA's rows
    const uint64_t qdims[4] = {(uint64_t)D, (uint64_t)p.n_q, (uint64_t)p.n_tok, (uint64_t)batch};
    const uint64_t qstrides[3] = {(uint64_t)D * 2, (uint64_t)p.n_q * D * 2,
                                  (uint64_t)p.n_tok * p.n_q * D * 2};
    const uint32_t qbox[4] = {64, (uint32_t)p.G, (uint32_t)(128 / p.G), 1};
    if (!encode_bf16_sw128(&qm, p.q, 4, qdims, qstrides, qbox)) return cudaErrorInvalidValue;
    MergeParams mp{};
    mp.tp = tree;
    mp.batch = batch;
    mp.n_rt = (p.n_tok * p.G + kTpRows - 1) / kTpRows;
    mp.workers = workers;
    mp.keys = kTpKeys;
    if (DEAL == kTreeShares) {
        const TpScratch ws = tp_scratch(batch, workers);
        uint8_t* base = static_cast<uint8_t*>(workspace);
        mp.part_o = reinterpret_cast<float*>(base);
        mp.part_ml = reinterpret_cast<float2*>(base + ws.ml_off);
        mp.before = reinterpret_cast<int32_t*>(base + ws.before_off);
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, km, vm, qm, mp);
    return e == cudaSuccess && DEAL == kTreeShares ? launch_tree_merge(mp, D, kTpRows, st) : e;
}

}  // namespace

size_t tree_pair_workspace(int batch, int workers) { return tp_scratch(batch, workers).bytes; }

template <int D>
static cudaError_t launch_tp_deal(const TreeParams& tp, int batch, void* workspace, int workers, int deal,
                                  cudaStream_t st) {
    const bool cap = tp.p.softcap > 0.f;
    switch (deal) {
        case kTreeShares:
            return cap ? launch_tp<D, true, kTreeShares>(tp, batch, workspace, workers, st)
                       : launch_tp<D, false, kTreeShares>(tp, batch, workspace, workers, st);
        case kTreeAlone:
            return cap ? launch_tp<D, true, kTreeAlone>(tp, batch, workspace, workers, st)
                       : launch_tp<D, false, kTreeAlone>(tp, batch, workspace, workers, st);
    }
    return cap ? launch_tp<D, true, kTreeWhole>(tp, batch, workspace, workers, st)
               : launch_tp<D, false, kTreeWhole>(tp, batch, workspace, workers, st);
}

cudaError_t launch_tree_pair(const TreeParams& tp, int head_dim, int batch, void* workspace,
                             int workers, int deal, cudaStream_t st) {
    if (head_dim == 256) return launch_tp_deal<256>(tp, batch, workspace, workers, deal, st);
    if (head_dim == 512) return launch_tp_deal<512>(tp, batch, workspace, workers, deal, st);
    return cudaErrorInvalidValue;
}

}  // namespace gemma
