// tree_attn.cu -- attention of a tree of drafted tokens over a device-resident KV cache.
//
// A sequence's tree has n nodes whose K/V rows were appended at base .. base + n - 1 (base = len -
// n). Node i stands at text position base + depth(i) and attends
//   the prefix keys j < base (on a sliding layer those with base + depth(i) - j < window), and
//   its ancestors and itself (on a sliding layer those with depth(i) - depth(m) < window);
// out = softmax(scale * q k^T) v over them. Definition and layers as in rows_attn.cu ("Porting
// Gemma-4 (2B / 4B / 12B) to AWS Inferentia2", sections 2.1-2.3 and 4.3).
//
// All nodes share the prefix, so a KV head's rows (nodes x G query heads) go through its keys
// together: with R rows a key costs 4 R d operations for 4 d bytes. Many rows run on the 5th-generation
// tensor cores (tree_tc.cu, tree_pair.cu). Here:
//  - tree_keys_kernel, head_dim 64 and 128, up to 16 rows, many keys: bound by memory. A warp has the 16
//    rows and a share of every tile's keys, and keeps O whole, so that no warp waits for another;
//  - tree_rows_kernel, head_dim 512, up to 32 rows: O of 16 rows is two warps' registers at least, so the
//    warps of a row group share out the keys of S and the columns of O += P V, with an exchange of row
//    maxima and one of P through shared memory per tile;
//  - tree_f32_kernel, the fp32 debug path.
// The first two, per CTA: one KV head of one sequence and one chunk of keys. A producer warp streams K and
// V tiles of 64 keys through a ring of slots (tiled TMA, 128-byte swizzle); mma.sync m16n8k16; the
// reference of a row's exponentials moves only when the maximum grows by more than 2^8; ancestor sets are
// four words per token, walked up from the parents while the first tiles load; only tiles that reach the
// tree or a window's edge look at masks. Sums, maxima and O are fp32; P is rounded to bf16 for the matrix
// instruction and summed as rounded. Chunks leave partial (m, l, O) for tree_combine_kernel, an unsplit
// launch writes `out`.
#include <atomic>
#include <climits>

#include "common.cuh"
#include "tc.cuh"
#include "tmap.h"
#include "tree.h"
#include "tree_dev.cuh"

namespace gemma {

namespace {

constexpr int kTrWarps = 8;                       // consumers
constexpr int kTrThreads = (kTrWarps + 1) * 32;
constexpr int T = kTreeKeyTile;
constexpr int kTrMaxSlots = 8;

// Shared memory: ring of key or value tiles, Q rows, P rows, row maxima, the tree.
template <int D, int MW>
struct TrLay {
    static constexpr int M = 16 * MW;             // rows of the tile
    static constexpr int CW = kTrWarps / MW;      // warps of a row group
    static constexpr int SLOT = T * D * 2;
    static constexpr int BOX = T * 128;           // one TMA box: 64 keys x 64 columns
    static constexpr int Q_ROW = 2 * D + 16;      // padded bytes per Q row
    static constexpr int P_ROW = 2 * T + 16;
    static constexpr int FIXED = M * Q_ROW + M * P_ROW + CW * M * 4 + 32 * kTrWords * 4 + 32 * 4 +
                                 kTreeMaxNodes * 4 + 2 * kTrMaxSlots * 8 + 1024;
    static constexpr int FIT = (227 * 1024 - FIXED) / SLOT;  // one CTA per SM
    static constexpr int SLOTS = FIT > kTrMaxSlots ? kTrMaxSlots : FIT;
    static constexpr int Q_OFF = SLOTS * SLOT;
    static constexpr int P_OFF = Q_OFF + M * Q_ROW;
    static constexpr int MAX_OFF = P_OFF + M * P_ROW;
    static constexpr int ANC_OFF = MAX_OFF + CW * M * 4;
    static constexpr int DEPTH_OFF = ANC_OFF + 32 * kTrWords * 4;
    static constexpr int PAR_OFF = DEPTH_OFF + 32 * 4;
    static constexpr int BAR_OFF = PAR_OFF + kTreeMaxNodes * 4;
    static constexpr int SMEM = BAR_OFF + 2 * kTrMaxSlots * 8 + 1024;  // + alignment slack
    static_assert(SLOTS >= 2 && SMEM <= 232448 && BAR_OFF % 8 == 0, "shared memory budget");
};

// The same for head_dim up to 128, where a warp holds O of its 16 rows whole: KG warps share out a tile's
// keys.
template <int D>
struct TrKeys {
    static constexpr int M = 16;                  // rows of the tile
    static constexpr int KG = 4;
    static constexpr int WARPS = KG;              // consumers
    static constexpr int SLOT = T * D * 2;
    static constexpr int Q_ROW = 2 * D + 16;
    static constexpr int O_ROW = D + 8;           // floats per row of the merge buffer
    static constexpr int MERGE = KG * M * O_ROW * 4;  // in the ring, once its tiles are used up
    static constexpr int FIXED = M * Q_ROW + 2 * KG * M * 4 + 32 * kTrWords * 4 + 32 * 4 +
                                 kTreeMaxNodes * 4 + 2 * kTrMaxSlots * 8 + 1024;
    static constexpr int FIT = (113 * 1024 - FIXED) / SLOT;  // two CTAs per SM
    static constexpr int SLOTS = FIT > kTrMaxSlots ? kTrMaxSlots : FIT;
    static constexpr int RING = SLOTS * SLOT;
    static constexpr int Q_OFF = RING;
    static constexpr int ML_OFF = Q_OFF + M * Q_ROW;                 // m [KG][M], l [KG][M]
    static constexpr int ANC_OFF = ML_OFF + 2 * KG * M * 4;
    static constexpr int DEPTH_OFF = ANC_OFF + 32 * kTrWords * 4;
    static constexpr int PAR_OFF = DEPTH_OFF + 32 * 4;
    static constexpr int BAR_OFF = PAR_OFF + kTreeMaxNodes * 4;
    static constexpr int SMEM = BAR_OFF + 2 * kTrMaxSlots * 8 + 1024;  // + alignment slack
    static_assert(SLOTS >= 4 && RING >= MERGE && SMEM <= 113 * 1024 && BAR_OFF % 8 == 0,
                  "shared memory budget");
};

// Byte offset of element (key, d) in a tile written by TMA with 128-byte swizzle.
GEMMA_DEVINL uint32_t tr_off(int key, int d) {
    return (uint32_t)((d >> 6) * (T * 128) + key * 128 + ((((d >> 3) & 7) ^ (key & 7)) << 4) +
                      (d & 7) * 2);
}

}  // namespace

// head_dim up to 128: a warp has the rows and a share of every tile's keys, and keeps O whole
template <int D>
__global__ void __launch_bounds__((TrKeys<D>::WARPS + 1) * 32, 2)
    tree_keys_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const TreeParams tp) {
    pdl_launch_dependents();
    using Lay = TrKeys<D>;
    constexpr int M = Lay::M, KG = Lay::KG, S = Lay::SLOTS, WARPS = Lay::WARPS;
    constexpr int KN = T / KG;       // a warp's keys of a tile
    constexpr int NT = KN / 8;
    constexpr int ON = D / 8;
    const RowsParams& p = tp.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem;
    uint8_t* sQ = smem + Lay::Q_OFF;
    float* sM = reinterpret_cast<float*>(smem + Lay::ML_OFF);                  // [KG][M]
    float* sL = sM + KG * M;                                                   // [KG][M]
    uint32_t* sAnc = reinterpret_cast<uint32_t*>(smem + Lay::ANC_OFF);         // [32][kTrWords]
    int* sDepth = reinterpret_cast<int*>(smem + Lay::DEPTH_OFF);               // [32]
    int* sPar = reinterpret_cast<int*>(smem + Lay::PAR_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
    uint64_t* empty = full + kTrMaxSlots;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int n_rows = p.n_tok * p.G;
    const bool direct = p.n_split == 1;

    pdl_wait();  // the previous kernel on the stream has completed
    const TrSeq sq = tr_seq(p, b);
    const int live = sq.bad ? 0 : max(0, min(n_rows, sq.n * p.G));  // rows of real nodes
    if (live == 0) {
        if (sq.bad && split == 0 && kvh == 0 && threadIdx.x == 0) report(p.err, sq.bad);
        for (int i = threadIdx.x; direct && i < n_rows * (D / 8); i += (WARPS + 1) * 32) {
            const int r = i / (D / 8), tk = r / p.G;
            __nv_bfloat16* dst =
                reinterpret_cast<__nv_bfloat16*>(p.out) +
                (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (r - tk * p.G)) * (size_t)D;
            reinterpret_cast<uint4*>(dst)[i - r * (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int first = tr_first(p, sq);
    const int kb = tr_start(p, sq) + split * p.chunk;
    if (kb >= sq.len) return;
    const int ke = min(sq.len, kb + p.chunk);
    const int n_tiles = (ke - kb + T - 1) / T;
    const int nops = p.k_eq_v ? 1 : 2;

    if (warp == WARPS) {
        // ------------------------- producer: tiles in the order of their use -------------------
        if (lane == 0) {
            for (int s = 0; s < S; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], WARPS);
            }
            fence_barrier_init();
        }
        __syncwarp();
        named_bar_arrive(1, (WARPS + 1) * 32);
        if (lane == 0) {
            const int n_loads = n_tiles * nops;
            int row3 = 0, slot0 = 0;
            bool ok = true;
            for (int L = 0; L < n_loads && ok; ++L) {
                const int s = L % S, use = L / S;
                if (use > 0 && !(ok = mbar_wait(&empty[s], (use - 1) & 1, p.err))) break;
                const bool is_v = nops == 2 && (L & 1);
                if (!is_v) {
                    const int t = nops == 2 ? L >> 1 : L;
                    if (!kv_place(p, b, kvh, kb + t * T, row3, slot0)) {
                        report(p.err, GEMMA_DEVERR_PAGE);  // reads zeros
                        row3 = p.n_pages * p.n_kv;
                    }
                }
                mbar_arrive_expect_tx(&full[s], Lay::SLOT);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(ring + s * Lay::SLOT + c * (T * 128), is_v ? &vmap : &kmap, c * 64,
                                slot0, row3, &full[s]);
            }
        }
        return;
    }

    // -------------------------------------- consumers ------------------------------------------
    // Q rows (zeros behind the tile's), and the tree
    {
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q);
        constexpr int CH = D / 8;
        for (int i = threadIdx.x; i < M * CH; i += WARPS * 32) {
            const int r = i / CH, ch = i - r * CH;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < live) {
                const int tk = r / p.G;
                v = __ldg(reinterpret_cast<const uint4*>(
                              q + (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (r - tk * p.G)) *
                                      (size_t)D) + ch);
            }
            *reinterpret_cast<uint4*>(sQ + r * Lay::Q_ROW + ch * 16) = v;
        }
    }
    bool bad = false;
    if ((int)threadIdx.x < sq.n) {
        const int m = __ldg(tp.parents + (size_t)b * p.n_tok + threadIdx.x);
        bad = m < -1 || m >= (int)threadIdx.x;
        sPar[threadIdx.x] = bad ? -1 : m;
    }
    bad = named_bar_or(2, WARPS * 32, bad);  // a bad tree: every row masked, zeros
    if (bad && split == 0 && kvh == 0 && threadIdx.x == 0)
        report(p.err, GEMMA_DEVERR_TREE);
    if ((int)threadIdx.x < (live - 1) / p.G + 1) {
        const int i = threadIdx.x;  // at most 32 tokens
        uint32_t set[kTrWords];
        sDepth[i] = tr_walk(sPar, i, p.is_sliding ? p.window : INT_MAX, set);
#pragma unroll
        for (int w = 0; w < kTrWords; ++w) sAnc[i * kTrWords + w] = set[w];
    }
    named_bar_sync(1, (WARPS + 1) * 32);  // with the producer: its barriers exist

    const int kg = warp;  // share of the keys
    const int g = lane >> 2, tq = lane & 3;
    // this thread's rows g and g + 8: the first prefix key they attend, and their token
    int lo[2], tok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = g + 8 * i;
        tok[i] = r < live && !bad ? r / p.G : -1;
        lo[i] = tok[i] < 0        ? INT_MAX
                : p.is_sliding ? max(0, sq.base + sDepth[tok[i]] - p.window + 1)
                                  : 0;
    }
    const int lo_max = max(lo[0], lo[1]);
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float o[ON][4];
#pragma unroll
    for (int j = 0; j < ON; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const uint32_t qa0 = smem_u32(sQ + ((lane & 15)) * Lay::Q_ROW + (lane >> 4) * 16);

    // No warp waits for another before the end: each has its own keys, and its rows' reference.
    bool ok = true;
    int L = 0;
    for (int t = 0; t < n_tiles; ++t) {
        const int kt0 = kb + t * T;
        const int sk = L % S;
        if (ok) ok = mbar_wait(&full[sk], (L / S) & 1, p.err);
        ++L;
        const uint8_t* tK = ring + sk * Lay::SLOT;

        // (1) S: 16 rows x this warp's keys
        float s[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t a0, a1, a2, a3;
            ldsm_x4(qa0 + ks * 32, a0, a1, a2, a3);
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                uint32_t b0, b1, b2, b3;
                const int key = kg * KN + j * 8 + (lane & 7) + ((lane >> 4) << 3);
                ldsm_x4(smem_u32(tK + tr_off(key, ks * 16 + ((lane >> 3) & 1) * 8)), b0, b1, b2, b3);
                mma_bf16(s[j], a0, a1, a2, a3, b0, b1);
                mma_bf16(s[j + 1], a0, a1, a2, a3, b2, b3);
            }
        }
        if (nops == 2) {  // K has been read
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[sk]);
        }

        // (2) scores, masks, the rows' maxima, P as the A operand of P V
        const int kw = kt0 + kg * KN;  // this warp's first key
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = tr_score(p, s[j][e]);
        if (!(kw >= lo_max && kw + KN <= sq.base)) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = kw + j * 8 + 2 * tq + (e & 1), i = e >> 1, m = key - sq.base;
                    bool in = m < 0 && key >= lo[i];
                    if (m >= 0 && key < ke && tok[i] >= 0)
                        in = (sAnc[tok[i] * kTrWords + (m >> 5)] >> (m & 31)) & 1u;
                    if (!in) s[j][e] = -INFINITY;
                }
        }
        float alpha[2];
        uint32_t pa[NT][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < NT; ++j) mx = fmax3f(mx, s[j][2 * i], s[j][2 * i + 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            alpha[i] = 1.f;
            if (mx > m_run[i] + kTrLazyLog2) {
                alpha[i] = fast_exp2(m_run[i] - mx);  // 0 while the reference is -inf
                m_run[i] = mx;
            }
            const float neg = m_run[i] == -INFINITY ? 0.f : -m_run[i];
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                pa[j][i] = pack_bf16(fast_exp2(s[j][2 * i] + neg), fast_exp2(s[j][2 * i + 1] + neg));
                sum += __uint_as_float(pa[j][i] << 16) + __uint_as_float(pa[j][i] & 0xffff0000u);
            }
            l_run[i] = fmaf(l_run[i], alpha[i], sum);
        }
        if (alpha[0] != 1.f || alpha[1] != 1.f) {
#pragma unroll
            for (int j = 0; j < ON; ++j) {
                o[j][0] *= alpha[0];
                o[j][1] *= alpha[0];
                o[j][2] *= alpha[1];
                o[j][3] *= alpha[1];
            }
        }

        // (3) O += P V over this warp's keys, all columns
        int sv = sk;
        if (nops == 2) {
            sv = L % S;
            if (ok) ok = mbar_wait(&full[sv], (L / S) & 1, p.err);
            ++L;
        }
        const uint8_t* tV = ring + sv * Lay::SLOT;
        const bool edge = kt0 < first || kt0 + T > ke;
#pragma unroll
        for (int kk = 0; kk < KN / 16; ++kk) {
            uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
            if (edge) {  // rows outside of the tree's keys may hold anything: zeros
                auto in = [&](int k) { return kw + k >= first && kw + k < ke; };
                const int k0 = kk * 16 + 2 * tq;
                mlo = (in(k0) ? 0x0000ffffu : 0u) | (in(k0 + 1) ? 0xffff0000u : 0u);
                mhi = (in(k0 + 8) ? 0x0000ffffu : 0u) | (in(k0 + 9) ? 0xffff0000u : 0u);
            }
            const int vkey = kg * KN + kk * 16 + (lane & 15);
#pragma unroll
            for (int j = 0; j < ON; j += 2) {
                uint32_t v0, v1, v2, v3;
                ldsm_x4_t(smem_u32(tV + tr_off(vkey, j * 8 + (lane >> 4) * 8)), v0, v1, v2, v3);
                mma_bf16(o[j], pa[2 * kk][0], pa[2 * kk][1], pa[2 * kk + 1][0], pa[2 * kk + 1][1],
                         v0 & mlo, v1 & mhi);
                mma_bf16(o[j + 1], pa[2 * kk][0], pa[2 * kk][1], pa[2 * kk + 1][0],
                         pa[2 * kk + 1][1], v2 & mlo, v3 & mhi);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[sv]);
    }

    // ---- merge of the key groups through the ring (its last tile has been read) ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 1);
        l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 2);
        if (tq == 0) {
            sM[kg * M + g + 8 * i] = m_run[i];
            sL[kg * M + g + 8 * i] = l_run[i];
        }
    }
    named_bar_sync(2, WARPS * 32);
    float* sO = reinterpret_cast<float*>(ring);  // [KG][M][O_ROW]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = g + 8 * i;
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < KG; ++k) top = fmaxf(top, sM[k * M + r]);
        const float w = m_run[i] == -INFINITY ? 0.f : fast_exp2(m_run[i] - top);
        float* dst = sO + (kg * M + r) * Lay::O_ROW + 2 * tq;
#pragma unroll
        for (int j = 0; j < ON; ++j)
            *reinterpret_cast<float2*>(dst + j * 8) =
                w == 0.f ? make_float2(0.f, 0.f) : make_float2(o[j][2 * i] * w, o[j][2 * i + 1] * w);
    }
    named_bar_sync(2, WARPS * 32);
    constexpr int CH = D / 4;  // four columns of a row per thread and step
    for (int x = threadIdx.x; x < n_rows * CH; x += WARPS * 32) {
        const int r = x / CH, ch = x - r * CH;
        float top = -INFINITY, l = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < KG; ++k) top = fmaxf(top, sM[k * M + r]);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(sO + (k * M + r) * Lay::O_ROW + 4 * ch);
            const float mk = sM[k * M + r];
            l += mk == -INFINITY ? sL[k * M + r] : fast_exp2(mk - top) * sL[k * M + r];  // (0, or NaN)
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
        if (direct) {
            const int tk = r / p.G;
            uint2* dst = reinterpret_cast<uint2*>(
                reinterpret_cast<__nv_bfloat16*>(p.out) +
                (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (r - tk * p.G)) * (size_t)D + 4 * ch);
            const float inv = 1.f / l;  // (no keys: zeros, whatever the other rows' V holds)
            *dst = l == 0.f ? make_uint2(0u, 0u)
                            : make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
        } else {
            const size_t pr =
                (((size_t)b * p.n_kv + kvh) * n_rows + r) * p.n_split + split;
            *reinterpret_cast<float4*>(p.o_part + pr * D + 4 * ch) = a;
            if (ch == 0) *reinterpret_cast<float2*>(p.ml_part + pr * 2) = make_float2(top, l);
        }
    }
}

// head_dim 512 (O of 16 rows is two warps' registers): the warps of a row group share out the keys of
// S and the columns of O
template <int D, int MW>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_rows_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const TreeParams tp) {
    pdl_launch_dependents();
    using Lay = TrLay<D, MW>;
    constexpr int M = Lay::M, CW = Lay::CW, S = Lay::SLOTS;
    constexpr int NT = T / CW / 8;   // 8-key n-tiles of a warp's share of S
    constexpr int OC = D / CW;       // a warp's columns of O
    constexpr int ON = OC / 8;
    const RowsParams& p = tp.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem;
    uint8_t* sQ = smem + Lay::Q_OFF;
    uint8_t* sP = smem + Lay::P_OFF;
    float* sMax = reinterpret_cast<float*>(smem + Lay::MAX_OFF);               // [CW][M]
    uint32_t* sAnc = reinterpret_cast<uint32_t*>(smem + Lay::ANC_OFF);         // [32][kTrWords]
    int* sDepth = reinterpret_cast<int*>(smem + Lay::DEPTH_OFF);               // [32]
    int* sPar = reinterpret_cast<int*>(smem + Lay::PAR_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
    uint64_t* empty = full + kTrMaxSlots;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int n_rows = p.n_tok * p.G;
    const bool direct = p.n_split == 1;

    pdl_wait();  // the previous kernel on the stream has completed
    const TrSeq sq = tr_seq(p, b);
    const int live = sq.bad ? 0 : max(0, min(n_rows, sq.n * p.G));  // rows of real nodes
    if (live == 0) {
        if (sq.bad && split == 0 && kvh == 0 && threadIdx.x == 0) report(p.err, sq.bad);
        for (int i = threadIdx.x; direct && i < n_rows * (D / 8); i += kTrThreads) {
            const int r = i / (D / 8), tk = r / p.G;
            __nv_bfloat16* dst =
                reinterpret_cast<__nv_bfloat16*>(p.out) +
                (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (r - tk * p.G)) * (size_t)D;
            reinterpret_cast<uint4*>(dst)[i - r * (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int first = tr_first(p, sq);
    const int kb = tr_start(p, sq) + split * p.chunk;
    if (kb >= sq.len) return;
    const int ke = min(sq.len, kb + p.chunk);
    const int n_tiles = (ke - kb + T - 1) / T;
    const int nops = p.k_eq_v ? 1 : 2;

    if (warp == kTrWarps) {
        // ------------------------- producer: tiles in the order of their use -------------------
        if (lane == 0) {
            for (int s = 0; s < S; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], kTrWarps);
            }
            fence_barrier_init();
        }
        __syncwarp();
        named_bar_arrive(1, kTrThreads);
        if (lane == 0) {
            const int n_loads = n_tiles * nops;
            int row3 = 0, slot0 = 0;
            bool ok = true;
            for (int L = 0; L < n_loads && ok; ++L) {
                const int s = L % S, use = L / S;
                if (use > 0 && !(ok = mbar_wait(&empty[s], (use - 1) & 1, p.err))) break;
                const bool is_v = nops == 2 && (L & 1);
                if (!is_v) {
                    const int t = nops == 2 ? L >> 1 : L;
                    if (!kv_place(p, b, kvh, kb + t * T, row3, slot0)) {
                        report(p.err, GEMMA_DEVERR_PAGE);  // reads zeros
                        row3 = p.n_pages * p.n_kv;
                    }
                }
                mbar_arrive_expect_tx(&full[s], Lay::SLOT);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(ring + s * Lay::SLOT + c * Lay::BOX, is_v ? &vmap : &kmap, c * 64,
                                slot0, row3, &full[s]);
            }
        }
        return;
    }

    // -------------------------------------- consumers ------------------------------------------
    // Q rows (zeros behind the tile's), and the tree
    {
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q);
        constexpr int CH = D / 8;
        for (int i = threadIdx.x; i < M * CH; i += kTrWarps * 32) {
            const int r = i / CH, ch = i - r * CH;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < live) {
                const int tk = r / p.G;
                v = __ldg(reinterpret_cast<const uint4*>(
                              q + (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (r - tk * p.G)) *
                                      (size_t)D) + ch);
            }
            *reinterpret_cast<uint4*>(sQ + r * Lay::Q_ROW + ch * 16) = v;
        }
    }
    bool bad = false;
    if ((int)threadIdx.x < sq.n) {
        const int m = __ldg(tp.parents + (size_t)b * p.n_tok + threadIdx.x);
        bad = m < -1 || m >= (int)threadIdx.x;
        sPar[threadIdx.x] = bad ? -1 : m;
    }
    bad = named_bar_or(2, kTrWarps * 32, bad);  // a bad tree: every row masked, zeros
    if (bad && split == 0 && kvh == 0 && threadIdx.x == 0)
        report(p.err, GEMMA_DEVERR_TREE);
    if ((int)threadIdx.x < (live - 1) / p.G + 1) {
        const int i = threadIdx.x;  // at most 32 tokens
        uint32_t set[kTrWords];
        sDepth[i] = tr_walk(sPar, i, p.is_sliding ? p.window : INT_MAX, set);
#pragma unroll
        for (int w = 0; w < kTrWords; ++w) sAnc[i * kTrWords + w] = set[w];
    }
    named_bar_sync(1, kTrThreads);  // with the producer: its barriers exist

    const int mw = warp / CW, cw = warp - mw * CW;  // row group, share of keys and columns
    const int g = lane >> 2, tq = lane & 3;
    // this thread's rows 16 mw + g and + 8: the first prefix key they attend, and their token
    int lo[2], tok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 16 * mw + g + 8 * i;
        tok[i] = r < live && !bad ? r / p.G : -1;
        lo[i] = tok[i] < 0        ? INT_MAX
                : p.is_sliding ? max(0, sq.base + sDepth[tok[i]] - p.window + 1)
                                  : 0;
    }
    const int lo_max = max(lo[0], lo[1]);
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float o[ON][4];
#pragma unroll
    for (int j = 0; j < ON; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    // A wait that gives up makes this warp stop waiting but keep walking the tiles, so that every
    // consumer warp still reaches every barrier.
    bool ok = true;
    int L = 0;
    for (int t = 0; t < n_tiles; ++t) {
        const int kt0 = kb + t * T;
        const int sk = L % S;
        if (ok) ok = mbar_wait(&full[sk], (L / S) & 1, p.err);
        ++L;
        const uint8_t* tK = ring + sk * Lay::SLOT;

        // (1) S: 16 rows x this warp's keys
        float s[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        const uint32_t qa0 =
            smem_u32(sQ + (16 * mw + (lane & 15)) * Lay::Q_ROW + (lane >> 4) * 16);
        if constexpr (NT == 1) {
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                uint32_t a[8], b0, b1, b2, b3;
                ldsm_x4(qa0 + ks * 64, a[0], a[1], a[2], a[3]);
                ldsm_x4(qa0 + ks * 64 + 32, a[4], a[5], a[6], a[7]);
                ldsm_x4(smem_u32(tK + tr_off(cw * 8 + (lane & 7), ks * 32 + (lane >> 3) * 8)), b0,
                        b1, b2, b3);
                mma_bf16(s[0], a[0], a[1], a[2], a[3], b0, b1);
                mma_bf16(s[0], a[4], a[5], a[6], a[7], b2, b3);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4(qa0 + ks * 32, a0, a1, a2, a3);
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t b0, b1, b2, b3;
                    const int key = cw * (8 * NT) + j * 8 + (lane & 7) + ((lane >> 4) << 3);
                    ldsm_x4(smem_u32(tK + tr_off(key, ks * 16 + ((lane >> 3) & 1) * 8)), b0, b1, b2,
                            b3);
                    mma_bf16(s[j], a0, a1, a2, a3, b0, b1);
                    mma_bf16(s[j + 1], a0, a1, a2, a3, b2, b3);
                }
            }
        }
        if (nops == 2) {  // K has been read
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[sk]);
        }

        // (2) scores, masks, the rows' maxima over all warps of the group
        const int kw = kt0 + cw * (8 * NT);  // this warp's first key
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = tr_score(p, s[j][e]);
        if (!(kw >= lo_max && kw + 8 * NT <= sq.base)) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = kw + j * 8 + 2 * tq + (e & 1), i = e >> 1, m = key - sq.base;
                    bool in = m < 0 && key >= lo[i];
                    if (m >= 0 && key < ke && tok[i] >= 0)
                        in = (sAnc[tok[i] * kTrWords + (m >> 5)] >> (m & 31)) & 1u;
                    if (!in) s[j][e] = -INFINITY;
                }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            mx[0] = fmax3f(mx[0], s[j][0], s[j][1]);
            mx[1] = fmax3f(mx[1], s[j][2], s[j][3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            if (tq == 0) sMax[cw * M + 16 * mw + g + 8 * i] = mx[i];
        }
        named_bar_sync(3 + mw, CW * 32);
        float alpha[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 16 * mw + g + 8 * i;
#pragma unroll
            for (int c = 0; c < CW; ++c) mx[i] = fmaxf(mx[i], sMax[c * M + r]);
            alpha[i] = 1.f;
            if (mx[i] > m_run[i] + kTrLazyLog2) {
                alpha[i] = fast_exp2(m_run[i] - mx[i]);  // 0 while the reference is -inf
                m_run[i] = mx[i];
            }
            const float neg = m_run[i] == -INFINITY ? 0.f : -m_run[i];
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t pb = pack_bf16(fast_exp2(s[j][2 * i] + neg),
                                              fast_exp2(s[j][2 * i + 1] + neg));
                *reinterpret_cast<uint32_t*>(sP + r * Lay::P_ROW +
                                             (cw * (8 * NT) + j * 8 + 2 * tq) * 2) = pb;
                sum += __uint_as_float(pb << 16) + __uint_as_float(pb & 0xffff0000u);
            }
            l_run[i] = fmaf(l_run[i], alpha[i], sum);
        }
        named_bar_sync(3 + mw, CW * 32);

        // (3) O = diag(alpha) O + P V over this warp's columns
        if (alpha[0] != 1.f || alpha[1] != 1.f) {
#pragma unroll
            for (int j = 0; j < ON; ++j) {
                o[j][0] *= alpha[0];
                o[j][1] *= alpha[0];
                o[j][2] *= alpha[1];
                o[j][3] *= alpha[1];
            }
        }
        int sv = sk;
        if (nops == 2) {
            sv = L % S;
            if (ok) ok = mbar_wait(&full[sv], (L / S) & 1, p.err);
            ++L;
        }
        const uint8_t* tV = ring + sv * Lay::SLOT;
        const bool edge = kt0 < first || kt0 + T > ke;
#pragma unroll
        for (int kk = 0; kk < T / 16; ++kk) {
            uint32_t a0, a1, a2, a3;
            ldsm_x4(smem_u32(sP + (16 * mw + (lane & 15)) * Lay::P_ROW + kk * 32 + (lane >> 4) * 16),
                    a0, a1, a2, a3);
            uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
            if (edge) {  // rows outside of the tree's keys may hold anything: zeros
                auto in = [&](int k) { return kt0 + k >= first && kt0 + k < ke; };
                const int k0 = kk * 16 + 2 * tq;
                mlo = (in(k0) ? 0x0000ffffu : 0u) | (in(k0 + 1) ? 0xffff0000u : 0u);
                mhi = (in(k0 + 8) ? 0x0000ffffu : 0u) | (in(k0 + 9) ? 0xffff0000u : 0u);
            }
            const int vkey = kk * 16 + (lane & 15);
#pragma unroll
            for (int j = 0; j < ON; j += 2) {
                uint32_t v0, v1, v2, v3;
                ldsm_x4_t(smem_u32(tV + tr_off(vkey, cw * OC + j * 8 + (lane >> 4) * 8)), v0, v1,
                          v2, v3);
                mma_bf16(o[j], a0, a1, a2, a3, v0 & mlo, v1 & mhi);
                mma_bf16(o[j + 1], a0, a1, a2, a3, v2 & mlo, v3 & mhi);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[sv]);
    }

    // ---- the rows' sums over the group's keys, and the results ----
    named_bar_sync(3 + mw, CW * 32);  // the last maxima have been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 1);
        l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 2);
        if (tq == 0) sMax[cw * M + 16 * mw + g + 8 * i] = l_run[i];
    }
    named_bar_sync(3 + mw, CW * 32);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 16 * mw + g + 8 * i;
        if (r >= n_rows) continue;
        float l = 0.f;
#pragma unroll
        for (int c = 0; c < CW; ++c) l += sMax[c * M + r];
        if (direct) {
            const int tk = r / p.G;
            __nv_bfloat16* dst =
                reinterpret_cast<__nv_bfloat16*>(p.out) +
                (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (r - tk * p.G)) * (size_t)D +
                cw * OC + 2 * tq;
            const float inv = 1.f / l;
#pragma unroll
            for (int j = 0; j < ON; ++j)  // (no keys: zeros, whatever the other rows' V holds)
                *reinterpret_cast<uint32_t*>(dst + j * 8) =
                    l == 0.f ? 0u : pack_bf16(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
        } else {
            const size_t pr =
                (((size_t)b * p.n_kv + kvh) * n_rows + r) * p.n_split + split;
            float* dst = p.o_part + pr * D + cw * OC + 2 * tq;
#pragma unroll
            for (int j = 0; j < ON; ++j)
                *reinterpret_cast<float2*>(dst + j * 8) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
            if (cw == 0 && tq == 0)
                *reinterpret_cast<float2*>(p.ml_part + pr * 2) = make_float2(m_run[i], l);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// merge of the chunks: M = max_c m_c, out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c
// ---------------------------------------------------------------------------------------------
// One warp per row and slice of 128 columns (64 at head_dim 64).
template <int D>
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeParams tp, long long n_warps) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    constexpr int V = D >= 128 ? 4 : 2, SL = D / (32 * V);
    const RowsParams& p = tp.p;
    const int lane = threadIdx.x & 31;
    const long long wi = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (wi >= n_warps) return;
    const long long row = wi / SL;
    const int col = (int)(wi - row * SL) * (32 * V) + lane * V;
    const int rows_total = p.n_tok * p.G;
    const int R = (int)(row % rows_total);
    const int kvh = (int)(row / rows_total % p.n_kv), b = (int)(row / rows_total / p.n_kv);
    const int tk = R / p.G;
    const TrSeq sq = tr_seq(p, b);
    const int nc = sq.bad || tk >= sq.n ? 0 : tr_chunks(p, sq);
    float acc[V], top = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    const float2* ml = reinterpret_cast<const float2*>(p.ml_part) + row * p.n_split;
    for (int c = lane; c < nc; c += 32) top = fmaxf(top, ml[c].x);
    top = warp_max(top);
    const float* src = p.o_part + row * p.n_split * D + col;
#pragma unroll 4
    for (int c = 0; c < nc; ++c) {
        const float2 mlc = ml[c];
        const float w = mlc.x == -INFINITY ? 0.f : fast_exp2(mlc.x - top);
        l = fmaf(w, mlc.y, l);
        if constexpr (V == 4) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(src + (size_t)c * D));
            acc[0] = fmaf(w, v.x, acc[0]);
            acc[1] = fmaf(w, v.y, acc[1]);
            acc[2] = fmaf(w, v.z, acc[2]);
            acc[3] = fmaf(w, v.w, acc[3]);
        } else {
            const float2 v = __ldcs(reinterpret_cast<const float2*>(src + (size_t)c * D));
            acc[0] = fmaf(w, v.x, acc[0]);
            acc[1] = fmaf(w, v.y, acc[1]);
        }
    }
    const float inv = 1.f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(
        reinterpret_cast<__nv_bfloat16*>(p.out) +
        (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (R - tk * p.G)) * (size_t)D + col);
#pragma unroll
    for (int e = 0; e < V; e += 2) dst[e / 2] = l == 0.f ? 0u : pack_bf16(acc[e] * inv, acc[e + 1] * inv);
}

// ---------------------------------------------------------------------------------------------
// fp32 (debug path): FFMA and expf
// ---------------------------------------------------------------------------------------------
// One CTA per row. A key belongs to D / 16 lanes, 16 columns each, so that its dot product takes two to
// five shuffles; the lanes of a key are one of the CTA's streams, each with its own softmax over every
// n-th key, and the streams meet in shared memory. Latency bound on a few hundred keys: the rows of a
// stream's next key are on their way while it works on one (17 nodes x 4 heads, 700 keys, head_dim 128:
// 28 us with a warp per key and five shuffles for each).
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) tree_f32_kernel(const TreeParams tp) {
    pdl_launch_dependents();
    pdl_wait();  // the previous kernel on the stream has completed
    constexpr int LPK = D / 16, STREAMS = WARPS * 32 / LPK;
    const RowsParams& p = tp.p;
    __shared__ int s_par[kTreeMaxNodes];
    __shared__ uint32_t s_set[kTrWords];
    __shared__ int s_depth;
    __shared__ __align__(16) float s_o[STREAMS][D];
    __shared__ float s_m[STREAMS], s_l[STREAMS];
    const int head = blockIdx.x % p.n_q, node = blockIdx.x / p.n_q, b = blockIdx.y;
    const int kvh = head / p.G;
    const TrSeq sq = tr_seq(p, b);
    float* out = reinterpret_cast<float*>(p.out) +
                 (((size_t)b * p.n_tok + node) * p.n_q + head) * (size_t)D;
    bool bad = false;
    if (!sq.bad && (int)threadIdx.x < sq.n) {
        const int m = __ldg(tp.parents + (size_t)b * p.n_tok + threadIdx.x);
        bad = m < -1 || m >= (int)threadIdx.x;
        s_par[threadIdx.x] = bad ? -1 : m;
    }
    bad = __syncthreads_or(bad);
    if (sq.bad || bad || node >= sq.n) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && (sq.bad || bad))
            report(p.err, sq.bad ? sq.bad : GEMMA_DEVERR_TREE);
        for (int c = threadIdx.x; c < D; c += WARPS * 32) out[c] = 0.f;
        return;
    }
    if (threadIdx.x == 0) {
        uint32_t set[kTrWords];
        s_depth = tr_walk(s_par, node, p.is_sliding ? p.window : INT_MAX, set);
#pragma unroll
        for (int w = 0; w < kTrWords; ++w) s_set[w] = set[w];
    }
    __syncthreads();
    const int lo = p.is_sliding ? max(0, sq.base + s_depth - p.window + 1) : 0;
    const int stream = threadIdx.x / LPK, part = threadIdx.x % LPK;  // columns 4 part + 4 LPK i ..
    const float4* q = reinterpret_cast<const float4*>(
        reinterpret_cast<const float*>(p.q) + (((size_t)b * p.n_tok + node) * p.n_q + head) * (size_t)D);
    const float4* K = reinterpret_cast<const float4*>(p.k);
    const float4* V = reinterpret_cast<const float4*>(p.v);
    const size_t rs = (size_t)kv_row_slots(p);
    float4 qr[4], acc[4], kn[4], vn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        qr[i] = __ldg(q + part + LPK * i);
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto attended = [&](int j) {
        const int n = j - sq.base;
        return n < 0 || ((s_set[n >> 5] >> (n & 31)) & 1u);
    };
    // the stream's first attended key from j on
    auto seek = [&](int j) {
        while (j < sq.len && !attended(j)) j += STREAMS;
        return j;
    };
    auto load = [&](int j) {
        int krow = 0, kslot = 0;
        const bool there = kv_place(p, b, kvh, j, krow, kslot);  // a bad page: zeros
        if (!there && part == 0) report(p.err, GEMMA_DEVERR_PAGE);
        const size_t at = ((size_t)krow * rs + (size_t)kslot) * (D / 4) + part;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kn[i] = there ? __ldg(K + at + LPK * i) : make_float4(0.f, 0.f, 0.f, 0.f);
            vn[i] = there ? __ldg(V + at + LPK * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    float m = -INFINITY, l = 0.f;
    int j = seek(lo + stream);
    if (j < sq.len) load(j);
    // (streams of a warp leave at different times: their shuffles name their own lanes)
    const unsigned mask = LPK == 32 ? 0xffffffffu
                                    : ((1u << (LPK & 31)) - 1) << (threadIdx.x % 32 / LPK * LPK);
    while (j < sq.len) {
        float s = 0.f;
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fmaf(qr[i].x, kn[i].x, s);
            s = fmaf(qr[i].y, kn[i].y, s);
            s = fmaf(qr[i].z, kn[i].z, s);
            s = fmaf(qr[i].w, kn[i].w, s);
            v[i] = vn[i];
        }
        j = seek(j + STREAMS);
        if (j < sq.len) load(j);
#pragma unroll
        for (int o = LPK / 2; o > 0; o >>= 1) s += __shfl_xor_sync(mask, s, o);
        s *= p.scale;
        if (p.softcap > 0.f) s = p.softcap * tanhf(s / p.softcap);
        if (!(s <= m)) {  // (a NaN too: it reaches the output)
            const float alpha = expf(m - s);
            m = s;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i].x *= alpha;
                acc[i].y *= alpha;
                acc[i].z *= alpha;
                acc[i].w *= alpha;
            }
        }
        const float w = s == -INFINITY ? 0.f : expf(s - m);
        l += w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[i].x = fmaf(w, v[i].x, acc[i].x);
            acc[i].y = fmaf(w, v[i].y, acc[i].y);
            acc[i].z = fmaf(w, v[i].z, acc[i].z);
            acc[i].w = fmaf(w, v[i].w, acc[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(s_o[stream])[part + LPK * i] = acc[i];
    if (part == 0) {
        s_m[stream] = m;
        s_l[stream] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
#pragma unroll 8
    for (int w = 0; w < STREAMS; ++w) top = fmaxf(top, s_m[w]);
    __syncthreads();
    if (threadIdx.x < STREAMS)  // the streams' weights in the place of their maxima
        s_m[threadIdx.x] = s_m[threadIdx.x] == -INFINITY ? 0.f : expf(s_m[threadIdx.x] - top);
    __syncthreads();
#pragma unroll 8
    for (int w = 0; w < STREAMS; ++w) sum = fmaf(s_m[w], s_l[w], sum);
    for (int c = threadIdx.x; c < D; c += WARPS * 32) {
        float x = 0.f;
#pragma unroll 8
        for (int w = 0; w < STREAMS; ++w)
            if (s_m[w] != 0.f) x = fmaf(s_o[w][c], s_m[w], x);
        out[c] = x / sum;
    }
}

// ---------------------------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------------------------
// The kernel of a shape: its layout, threads and entry.
template <int D, int MW>
struct TrKernel {
    using Lay = TrKeys<D>;
    static constexpr int THREADS = (Lay::WARPS + 1) * 32;
    static auto entry() { return tree_keys_kernel<D>; }
};
template <int MW>
struct TrKernel<512, MW> {
    using Lay = TrLay<512, MW>;
    static constexpr int THREADS = kTrThreads;
    static auto entry() { return tree_rows_kernel<512, MW>; }
};

int tree_ctas_per_sm(int head_dim) {
    return head_dim <= 128 ? 2 : 1;
}

template <int D, int MW>
static cudaError_t launch_rows_dm(const TreeParams& tp, int batch, cudaStream_t st) {
    using Lay = typename TrKernel<D, MW>::Lay;
    const RowsParams& p = tp.p;
    auto kernel = TrKernel<D, MW>::entry();
    static std::atomic<bool> configured[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_relaxed);
    }
    CUtensorMap km, vm;
    // [rows][slots][D]: rows = sequences x KV heads (pages x KV heads for a paged pool)
    const uint64_t slots = (uint64_t)(p.page_size ? p.page_size : p.cap);
    const uint64_t rows = (uint64_t)(p.page_size ? p.n_pages : batch) * p.n_kv;
    const uint64_t dims[3] = {(uint64_t)D, slots, rows};
    const uint64_t strides[2] = {(uint64_t)D * 2, slots * D * 2};
    const uint32_t box[3] = {64, (uint32_t)T, 1};
    if (!encode_bf16_sw128(&km, p.k, 3, dims, strides, box)) return cudaErrorInvalidValue;
    if (!encode_bf16_sw128(&vm, p.v, 3, dims, strides, box)) return cudaErrorInvalidValue;
    return launch_pdl(kernel, dim3(p.n_split, p.n_kv, batch), dim3(TrKernel<D, MW>::THREADS),
                      Lay::SMEM, st, km, vm, tp);
}

cudaError_t launch_tree_rows(const TreeParams& tp, int head_dim, int batch, cudaStream_t st) {
    const int rows = tp.p.n_tok * tp.p.G;
    if (rows > kTreeRowsMax || (head_dim != 512 && rows > 16)) return cudaErrorInvalidValue;
    switch (head_dim) {
        case 64: return launch_rows_dm<64, 1>(tp, batch, st);
        case 128: return launch_rows_dm<128, 1>(tp, batch, st);
        case 512:
            return rows <= 16 ? launch_rows_dm<512, 1>(tp, batch, st) : launch_rows_dm<512, 2>(tp, batch, st);
    }
    return cudaErrorInvalidValue;
}

template <int D>
static cudaError_t launch_f32_d(const TreeParams& tp, int batch, cudaStream_t st) {
    const dim3 grid((unsigned)(tp.p.n_tok * tp.p.n_q), batch);
    // a CTA per SM: twice the streams for it. 8 / 16 warps: 136 rows over 700 keys of head_dim 128 16.0 / 11.0
    // us, 48 over 1600 of 256 38 / 26; 272 over 700 of 128 16.8 / 20.0
    if ((long long)grid.x * batch <= tp.n_sm)
        return launch_pdl(tree_f32_kernel<D, 16>, grid, dim3(512), 0, st, tp);
    return launch_pdl(tree_f32_kernel<D, 8>, grid, dim3(256), 0, st, tp);
}

cudaError_t launch_tree_f32(const TreeParams& tp, int head_dim, int batch, cudaStream_t st) {
    switch (head_dim) {
        case 64: return launch_f32_d<64>(tp, batch, st);
        case 128: return launch_f32_d<128>(tp, batch, st);
        case 256: return launch_f32_d<256>(tp, batch, st);
        case 512: return launch_f32_d<512>(tp, batch, st);
    }
    return cudaErrorInvalidValue;
}

template <int D>
static cudaError_t launch_combine_d(const TreeParams& tp, int batch, cudaStream_t st) {
    constexpr int SL = D >= 128 ? D / 128 : 1;
    const long long warps = (long long)batch * tp.p.n_q * tp.p.n_tok * SL;
    return launch_pdl(tree_combine_kernel<D>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st,
                      tp, warps);
}

cudaError_t launch_tree_combine(const TreeParams& tp, int head_dim, int batch, cudaStream_t st) {
    switch (head_dim) {
        case 64: return launch_combine_d<64>(tp, batch, st);
        case 128: return launch_combine_d<128>(tp, batch, st);
        case 512: return launch_combine_d<512>(tp, batch, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gemma
