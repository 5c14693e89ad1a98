// q4_attn.cu -- attention of a few query rows over a 4-bit KV cache (format: q4.h).
//
// For the rows (token, query head) of one KV head of one sequence, with keys j of its mask:
//   S[j][r] = cap(scale * sum_g sk[j][g] * (codes_k[j] . q[r])_g),  P = 2^(S - m),
//   O[d][r] = sum_j P[j][r] sv[j][g(d)] codes_v[j][d],  out = O / sum_j P[j][r].
// Both products run on mma.sync m16n8k16 (fp16 in, fp32 sums) with the cache as the 16-row
// operand and the query rows as the 8-column one, so that up to 8 rows cost one instruction
// and 16 rows two. The codes go in as they are: rotr(word, 4j) & 0x80078007 is a pair of fp16
// numbers code * 2^-24. Scales never touch the codes: K's multiply the fp32 sums of a group of
// 64 elements, V's multiply P (a warp's output columns all lie in one group).
//
// A CTA takes 8 * NQ rows and one chunk of keys, 128 keys at a time: one thread streams code tiles
// (TMA, 128-byte swizzle for rows of at least 128 bytes) and scales (bulk copies) into a ring of
// stages; eight warps each take 16 keys of S over all of head_dim (the query fragments stay in
// registers), exchange P through shared memory (one barrier per tile) and take a 64-column group
// of O (at head_dim < 512 the warps of a group share out the tile's keys). There is no producer
// warp: a ninth warp would cost the other eight a third of their registers.
// The softmax reference m is common to the CTA and lazy: it moves only when a score exceeds it by
// more than 2^8, which the tile's one barrier votes on. P and its product with V's scale are
// rounded to fp16 (2^-11 each; the output is rounded to bf16, 2^-8); V's scales enter relative to
// the largest one of the chunk so far, scaled into [2^5, 2^6), so that the product stays in fp16's
// normal range down to 2^-20 of it. Everything else is fp32.
#include <cuda_fp16.h>

#include <atomic>
#include <climits>

#include "attn_internal.h"
#include "common.cuh"
#include "q4.h"
#include "tc.cuh"
#include "tmap.h"

namespace gemma {

namespace {

constexpr int kT = kQ4KeyTile;      // keys per tile
constexpr int kWarps = 8;           // warps per CTA
constexpr int kThreads = kWarps * 32;
constexpr int kMaxStages = 8;
constexpr float kLazyLog2 = 8.f;
constexpr uint32_t kPairMask = 0x80078007u;

struct Q4AttnParams {
    RowsParams r;  // shapes, masks, q / out / partials (k, v: the code arrays)
    const __nv_bfloat16* k_scales;
    const __nv_bfloat16* v_scales;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int j) {
    return __funnelshift_r(word, word, 4 * j) & kPairMask;
}
// Barrier of the CTA that also ORs a flag over its threads.
__device__ __forceinline__ bool cta_vote(bool flag) { return __syncthreads_or(flag) != 0; }

template <int D>
struct Q4Layout {
    static constexpr int NG = D / kQ4Group;                     // scale groups per row
    static constexpr int ROWB = D / 2;                          // code bytes per row
    static constexpr int BOXB = ROWB < 128 ? ROWB : 128;        // bytes per row of one TMA box
    static constexpr int CODES = kT * ROWB;                     // one tile of codes
    static constexpr int SCALES = kT * NG * 2;                  // and of scales
    static constexpr int OP = CODES + (SCALES + 1023) / 1024 * 1024;  // one operand of a stage
    static constexpr int O_STRIDE = D + 4;                      // fp32 words per output row
};

// Byte of a code tile at (key, byte x of its row); 128-byte swizzle where rows fill it.
template <int D>
__device__ __forceinline__ uint32_t code_off(int key, int x) {
    using L = Q4Layout<D>;
    if (L::BOXB < 128) return (uint32_t)(key * L::ROWB + x);
    return (uint32_t)((x >> 7) * (kT * 128) + key * 128 + ((((x >> 4) & 7) ^ (key & 7)) << 4) +
                      (x & 15));
}
// Key (of 8) that MMA row g of S stands for: with the swizzle, keys 2g % 8 + g / 4 keep the 8-byte
// reads of four rows by four lanes free of bank conflicts.
template <int D>
__device__ __forceinline__ int key_of_row(int g) {
    return Q4Layout<D>::BOXB < 128 ? g : (g & 3) * 2 + (g >> 2);
}

struct Range {
    int lo, hi;  // keys [lo, hi) of one row
};
__device__ __forceinline__ Range row_range(const RowsParams& p, int len, int R) {
    const int pos = len - p.n_tok + R / p.G;
    return Range{p.is_sliding ? max(0, pos - p.window + 1) : 0, pos + 1};
}
// First key of a row tile's chunks: its first row's first key, rounded down to where a tile may
// start (32 keeps scale rows 16-byte aligned; a tile must not wrap round a ring or leave a page).
__device__ __forceinline__ int tile_base(const RowsParams& p, int lo) {
    return lo & ~((p.ring || p.page_size ? kT : 32) - 1);
}
__device__ __forceinline__ bool bad_length(const RowsParams& p, int len) {
    return len < p.n_tok || (!p.ring && len > p.cap) || len > p.max_seq_len;
}

template <int D, int NQ, int MINB>
__global__ void __launch_bounds__(kThreads, MINB)
    q4_attn_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const Q4AttnParams pp) {
    pdl_launch_dependents();
    using L = Q4Layout<D>;
    constexpr int RT = 8 * NQ;
    constexpr int NG = L::NG;
    constexpr int KSP = kWarps / NG;   // warps that share a column group
    constexpr int KW = kT / KSP;       // keys per warp of a tile in P V
    const RowsParams& p = pp.r;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kMaxStages];
    __shared__ __align__(16) __half sP[2][NQ][kT][8];
    __shared__ __align__(16) __half sV[kWarps][KW];
    __shared__ float sMax[kWarps][RT], sSum[kWarps][RT];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % p.n_split, rt = blockIdx.x / p.n_split;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int rows_total = p.n_tok * p.G, row0 = rt * RT;
    const int n_rows = min(RT, rows_total - row0);
    const bool direct = p.n_split == 1;

    pdl_wait();
    const int len = p.seq_lens[b];
    if (bad_length(p, len)) {
        if (split == 0) {
            if (threadIdx.x == 0) report(p.err, GEMMA_DEVERR_SEQ_LEN);
            if (direct)
                for (int i = threadIdx.x; i < n_rows * (D / 8); i += kThreads) {
                    const int R = row0 + i / (D / 8), tok = R / p.G;
                    reinterpret_cast<uint4*>(p.out)[(((size_t)b * p.n_tok + tok) * p.n_q +
                                                     kvh * p.G + (R - tok * p.G)) * (D / 8) +
                                                    i % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
                }
        }
        return;
    }
    const Range first = row_range(p, len, row0), last = row_range(p, len, row0 + n_rows - 1);
    const int kb = tile_base(p, first.lo) + split * p.chunk;
    const int ke = min(last.hi, kb + p.chunk);
    if (kb >= ke) return;  // the combine pass skips it
    const int n_tiles = (ke - kb + kT - 1) / kT;
    const int nops = p.k_eq_v ? 1 : 2;
    const int stage_bytes = nops * L::OP;
    const int S = p.n_stages;

    // Loads of tile t into its stage (one thread). No empty barriers: when the warps have voted on
    // tile t, every one of them has finished with tile t - 1, whose stage is then refilled.
    auto load_tile = [&](int t) {
        const int slots = kv_row_slots(p);
        uint64_t* bar = &full[t % S];
        uint8_t* st = smem + (t % S) * stage_bytes;
        int row = 0, slot = 0;
        const bool ok = kv_place(p, b, kvh, kb + t * kT, row, slot);
        // scale rows that exist (a tile may reach behind the last slot; capacities and tile starts
        // are multiples of 32, so the copies stay multiples of 16 bytes)
        const uint32_t sbytes = ok ? (uint32_t)(min(kT, slots - slot) * NG * 2) : 0u;
        if (!ok) {  // a bad page reads as zeros
            report(p.err, GEMMA_DEVERR_PAGE);
            row = p.n_pages * p.n_kv;
            for (int o = 0; o < nops; ++o)
                for (int i = 0; i < L::SCALES / 16; ++i)
                    reinterpret_cast<uint4*>(st + o * L::OP + L::CODES)[i] =
                        make_uint4(0u, 0u, 0u, 0u);
        }
        mbar_arrive_expect_tx(bar, (uint32_t)nops * (L::CODES + sbytes));
        for (int o = 0; o < nops; ++o) {
            uint8_t* dst = st + o * L::OP;
#pragma unroll
            for (int c = 0; c < L::ROWB / L::BOXB; ++c)
                tma_load_3d(dst + c * kT * 128, o ? &vmap : &kmap, c * 128, slot, row, bar);
            if (sbytes)
                bulk_g2s(dst + L::CODES,
                         (o ? pp.v_scales : pp.k_scales) + ((size_t)row * slots + slot) * NG,
                         sbytes, bar);
        }
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
        for (int t = 0; t < min(S, n_tiles); ++t) load_tile(t);
    }
    __syncwarp();

    const int g = lane >> 2, tq = lane & 3;
    // Query fragments: lane (g, tq) holds, of row g of each 8-row tile, elements 16 tq .. 16 tq + 15
    // of every group, the ones whose codes it reads. A row is scaled by a power of two that brings
    // its largest element into [2^13, 2^14) (exact unless an element is 2^-37 of that).
    uint32_t qf[NG * 4][NQ][2];
    float qscale[NQ];  // 2^-e of row g: score = sum * 2^24 / qscale * scale
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int R = row0 + n * 8 + g;
        uint4 raw[NG][2];
        uint32_t mx = 0;
        if (n * 8 + g < n_rows) {
            const int tok = R / p.G;
            const uint4* src = reinterpret_cast<const uint4*>(p.q) +
                               (((size_t)b * p.n_tok + tok) * p.n_q + kvh * p.G +
                                (R - tok * p.G)) * (D / 8) + 2 * tq;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                raw[i][0] = src[i * 8];
                raw[i][1] = src[i * 8 + 1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NG; ++i) raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {raw[i][h].x, raw[i][h].y, raw[i][h].z, raw[i][h].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
            }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // biased exponent of the largest element -> factor 2^(13 - (exponent - 127))
        const int ex = min(max((int)(mx >> 7), 13), 254);
        qscale[n] = __uint_as_float((uint32_t)(267 - ex) << 23);
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const uint4 v = raw[i][ks >> 1];
                const uint32_t w0 = ks & 1 ? v.z : v.x, w1 = ks & 1 ? v.w : v.y;
                qf[i * 4 + ks][n][0] = pack_f16(__uint_as_float(w0 << 16) * qscale[n],
                                                __uint_as_float(w0 & 0xffff0000u) * qscale[n]);
                qf[i * 4 + ks][n][1] = pack_f16(__uint_as_float(w1 << 16) * qscale[n],
                                                __uint_as_float(w1 & 0xffff0000u) * qscale[n]);
            }
    }
    // the rows whose scores this lane holds: 8 n + 2 tq + c
    float inv[NQ][2], m_run[NQ][2], l_run[NQ][2];
    int r_lo[NQ][2], r_hi[NQ][2];
    const float fac = p.softcap > 0.f ? p.cap_inner : p.scale_log2;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            inv[n][c] = fac / __shfl_sync(0xffffffffu, qscale[n], (2 * tq + c) * 4);
            m_run[n][c] = -INFINITY;
            l_run[n][c] = 0.f;
            const int r = n * 8 + 2 * tq + c;
            const Range rr = row_range(p, len, row0 + min(r, n_rows - 1));
            r_lo[n][c] = r < n_rows ? rr.lo : INT_MAX;
            r_hi[n][c] = min(rr.hi, ke);
        }
    float o[4][NQ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NQ; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    int v_exp = 6;  // biased exponent that V's scales are relative to
    const int wg = warp % NG, ksp = warp / NG;
    const int krow = warp * 16 + key_of_row<D>(g);  // this lane's keys of S: krow, krow + 8

    __syncthreads();
    bool ok = true;
    for (int t = 0; t < n_tiles; ++t) {
        const int s = t % S;
        if (ok) ok = mbar_wait(&full[s], (t / S) & 1, p.err);
        const uint8_t* tK = smem + s * stage_bytes;
        const uint8_t* tV = tK + (nops - 1) * L::OP;
        const int key0 = kb + t * kT;

        // (1) S of 16 keys
        float sv[NQ][4];
#pragma unroll
        for (int n = 0; n < NQ; ++n) sv[n][0] = sv[n][1] = sv[n][2] = sv[n][3] = 0.f;
        {
            const __nv_bfloat16* sk = reinterpret_cast<const __nv_bfloat16*>(tK + L::CODES);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const uint2 wa =
                    *reinterpret_cast<const uint2*>(tK + code_off<D>(krow, i * 32 + tq * 8));
                const uint2 wb =
                    *reinterpret_cast<const uint2*>(tK + code_off<D>(krow + 8, i * 32 + tq * 8));
                float acc[NQ][4];
#pragma unroll
                for (int n = 0; n < NQ; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint32_t xa = ks < 2 ? wa.x : wa.y, xb = ks < 2 ? wb.x : wb.y;
                    const int j = 2 * (ks & 1);
                    const uint32_t a0 = code_pair(xa, j), a1 = code_pair(xb, j);
                    const uint32_t a2 = code_pair(xa, j + 1), a3 = code_pair(xb, j + 1);
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        mma_f16(acc[n], a0, a1, a2, a3, qf[i * 4 + ks][n][0], qf[i * 4 + ks][n][1]);
                }
                const float ska = __bfloat162float(sk[krow * NG + i]);
                const float skb = __bfloat162float(sk[(krow + 8) * NG + i]);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    sv[n][0] = fmaf(acc[n][0], ska, sv[n][0]);
                    sv[n][1] = fmaf(acc[n][1], ska, sv[n][1]);
                    sv[n][2] = fmaf(acc[n][2], skb, sv[n][2]);
                    sv[n][3] = fmaf(acc[n][3], skb, sv[n][3]);
                }
            }
        }
        // scores in log2 units, masked keys -inf
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = k & 1, key = key0 + krow + 8 * (k >> 1);
                float x = sv[n][k] * 16777216.f * inv[n][c];
                if (p.softcap > 0.f) x = p.cap_log2 * tanhf(x);
                x = key >= r_lo[n][c] && key < r_hi[n][c] ? x : -INFINITY;
                sv[n][k] = x;
                grow = grow || x > m_run[n][c] + kLazyLog2;
            }
        __half(*P)[kT][8] = sP[t & 1];
        float pr[NQ][4];
        auto exponentiate = [&]() {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float m = m_run[n][k & 1];
                    pr[n][k] = fast_exp2(sv[n][k] - (m == -INFINITY ? 0.f : m));
                }
                *reinterpret_cast<uint32_t*>(&P[n][krow][2 * tq]) = pack_f16(pr[n][0], pr[n][1]);
                *reinterpret_cast<uint32_t*>(&P[n][krow + 8][2 * tq]) = pack_f16(pr[n][2], pr[n][3]);
            }
        };
        exponentiate();
        // V's scales of this warp's keys and group, as fp16 relative to 2^v_exp
        {
            const __nv_bfloat16* vs = reinterpret_cast<const __nv_bfloat16*>(tV + L::CODES);
            uint32_t sb[(KW + 31) / 32], mx = 0;
#pragma unroll
            for (int i = 0; i < (KW + 31) / 32; ++i) {
                const int k = i * 32 + lane, key = key0 + ksp * KW + k;
                sb[i] = 0;
                if (k < KW && key >= first.lo && key < ke)
                    sb[i] = __bfloat16_as_ushort(vs[(ksp * KW + k) * NG + wg]);
                if (sb[i] < 0x7f80u) mx = max(mx, sb[i]);
            }
            mx = __reduce_max_sync(0xffffffffu, mx) >> 7;
            if ((int)mx > v_exp) {
                const float a = v_exp - (int)mx < -126
                                    ? 0.f
                                    : __uint_as_float((uint32_t)(127 + v_exp - (int)mx) << 23);
                v_exp = (int)mx;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[i][n][k] *= a;
            }
            const float f = __uint_as_float((uint32_t)(259 - v_exp) << 23);  // 2^(5 - (v_exp - 127))
#pragma unroll
            for (int i = 0; i < (KW + 31) / 32; ++i)
                if (i * 32 + lane < KW)
                    sV[warp][i * 32 + lane] = __float2half_rn(__uint_as_float(sb[i] << 16) * f);
        }
        const bool moved = cta_vote(grow);
        if (threadIdx.x == 0 && t > 0 && t - 1 + S < n_tiles) load_tile(t - 1 + S);
        __syncwarp();
        if (moved) {
            // the reference moves: the rows' maxima over the CTA's warps, P anew
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = fmaxf(sv[n][c], sv[n][c + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                    if (g == 0) sMax[warp][n * 8 + 2 * tq + c] = mx;
                }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = m_run[n][c];
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sMax[w][n * 8 + 2 * tq + c]);
                    if (mx > m_run[n][c]) {
                        const float a = fast_exp2(m_run[n][c] - mx);  // 0 from -inf
                        m_run[n][c] = mx;
                        l_run[n][c] *= a;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[i][n][c] *= a;
                            o[i][n][c + 2] *= a;
                        }
                    }
                }
            exponentiate();
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) l_run[n][c] += pr[n][c] + pr[n][c + 2];

        // (2) O of 64 columns over this warp's keys
#pragma unroll 2
        for (int kk = 0; kk < KW; kk += 16) {
            const int kt = ksp * KW + kk;
            uint32_t bf[NQ][2];
            if (NQ == 2) {
                const uint32_t a = smem_u32(&P[lane >> 4][kt + (lane & 15)][0]);
                ldsm_x4_t(a, bf[0][0], bf[0][1], bf[NQ - 1][0], bf[NQ - 1][1]);
            } else {
                const uint32_t a = smem_u32(&P[0][kt + (lane & 15)][0]);
                asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                             : "=r"(bf[0][0]), "=r"(bf[0][1])
                             : "r"(a));
            }
            const uint32_t s0 = *reinterpret_cast<const uint32_t*>(&sV[warp][kk + 2 * tq]);
            const uint32_t s1 = *reinterpret_cast<const uint32_t*>(&sV[warp][kk + 2 * tq + 8]);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                bf[n][0] = mul_f16x2(bf[n][0], s0);
                bf[n][1] = mul_f16x2(bf[n][1], s1);
            }
            uint32_t w[4];  // words of keys 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9: columns 8 g .. 8 g + 7
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = *reinterpret_cast<const uint32_t*>(
                    tV + code_off<D>(kt + 2 * tq + (k & 1) + 8 * (k >> 1), wg * 32 + g * 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // MMA rows g, g + 8: columns 8 g + 2 i, 8 g + 2 i + 1
                const uint32_t r0 = code_pair(w[0], i), r1 = code_pair(w[1], i);
                const uint32_t r2 = code_pair(w[2], i), r3 = code_pair(w[3], i);
                const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
                const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
#pragma unroll
                for (int n = 0; n < NQ; ++n) mma_f16(o[i][n], a0, a1, a2, a3, bf[n][0], bf[n][1]);
            }
        }
        __syncwarp();
    }

    // ------------------------------------ epilogue -------------------------------------------
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float l = l_run[n][c];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
            if (g == 0) {
                sSum[warp][n * 8 + 2 * tq + c] = l;
                if (warp == 0) sMax[0][n * 8 + 2 * tq + c] = m_run[n][c];
            }
        }
    __syncthreads();  // every tile consumed: the stages are free
    float* sO = reinterpret_cast<float*>(smem);  // [KSP][RT][O_STRIDE]
    const float f2 = __uint_as_float((uint32_t)(v_exp - 5) << 23);  // 2^(v_exp - 127 - 5)
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float* dst = sO + ((size_t)ksp * RT + n * 8 + 2 * tq + c) * L::O_STRIDE + wg * 64 + g * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float2*>(dst + 2 * i) =
                    make_float2(o[i][n][c] * 16777216.f * f2, o[i][n][c + 2] * 16777216.f * f2);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < n_rows * (D / 8); i += kThreads) {
        const int r = i / (D / 8), x = (i - r * (D / 8)) * 8;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll
        for (int h = 0; h < KSP; ++h)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += sO[((size_t)h * RT + r) * L::O_STRIDE + x + k];
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += sSum[w][r];
        const int R = row0 + r;
        if (direct) {
            const int tok = R / p.G;
            const float il = 1.f / l;
            reinterpret_cast<uint4*>(p.out)[((((size_t)b * p.n_tok + tok) * p.n_q + kvh * p.G +
                                              (R - tok * p.G)) * D + x) / 8] =
                make_uint4(pack_bf16(v[0] * il, v[1] * il), pack_bf16(v[2] * il, v[3] * il),
                           pack_bf16(v[4] * il, v[5] * il), pack_bf16(v[6] * il, v[7] * il));
        } else {
            const size_t pr = (((size_t)b * p.n_kv + kvh) * rows_total + R) * p.n_split + split;
            float4* dst = reinterpret_cast<float4*>(p.o_part + pr * D + x);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            if (x == 0) {
                p.ml_part[2 * pr] = sMax[0][r];
                p.ml_part[2 * pr + 1] = l;
            }
        }
    }
}

// Merge of a row's chunks: M = max m_c, out = sum 2^(m_c - M) O_c / sum 2^(m_c - M) l_c. One CTA
// per row; thread groups share out the chunks and meet in shared memory, in a fixed order.
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) q4_merge_kernel(const RowsParams p, int row_tile) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int TPG = D / 4, NGRP = kMergeThreads / TPG;
    __shared__ float s_w[kQ4MaxSplit];
    __shared__ float4 s_red[kMergeThreads];
    __shared__ float s_inv;
    const int rows_total = p.n_tok * p.G;
    const int R = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int tok = R / p.G, head = kvh * p.G + R - tok * p.G, tid = threadIdx.x;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                         (((size_t)b * p.n_tok + tok) * p.n_q + head) * D;
    const int len = p.seq_lens[b];
    if (bad_length(p, len)) {
        for (int c = tid; c < D; c += kMergeThreads) dst[c] = __float2bfloat16_rn(0.f);
        return;
    }
    const int row0 = R / row_tile * row_tile;
    const Range first = row_range(p, len, row0);
    const Range last = row_range(p, len, min(row0 + row_tile, rows_total) - 1);
    const int nc = min(p.n_split, (last.hi - tile_base(p, first.lo) + p.chunk - 1) / p.chunk);
    const size_t base = (((size_t)b * p.n_kv + kvh) * rows_total + R) * p.n_split;
    if (tid < 32) {
        float m[kQ4MaxSplit / 32], l[kQ4MaxSplit / 32], M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < kQ4MaxSplit / 32; ++i) {
            const int c = tid + 32 * i;
            m[i] = c < nc ? p.ml_part[(base + c) * 2] : -INFINITY;
            l[i] = c < nc ? p.ml_part[(base + c) * 2 + 1] : 0.f;
            M = fmaxf(M, m[i]);
        }
        M = warp_max(M);
#pragma unroll
        for (int i = 0; i < kQ4MaxSplit / 32; ++i) {
            // a chunk without keys of this row has m = -inf and no weight
            const float w = m[i] == -INFINITY ? 0.f : exp2f(m[i] - M);
            s_w[tid + 32 * i] = w;
            sum = fmaf(w, l[i], sum);
        }
        sum = warp_sum(sum);
        if (tid == 0) s_inv = 1.f / sum;
    }
    __syncthreads();
    const int grp = tid / TPG, c4 = tid - grp * TPG;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = grp; c < nc; c += NGRP) {
        const float w = s_w[c];
        const float4 v = *reinterpret_cast<const float4*>(p.o_part + (base + c) * D + c4 * 4);
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
    }
    s_red[tid] = acc;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int h = 1; h < NGRP; ++h) {
            const float4 u = s_red[h * TPG + c4];
            acc.x += u.x;
            acc.y += u.y;
            acc.z += u.z;
            acc.w += u.w;
        }
        const float inv = s_inv;
        *reinterpret_cast<uint2*>(dst + c4 * 4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
}

// uint8 tensor map over [rows][slots][row bytes]
bool encode_codes(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t slots,
                  uint64_t rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {row_bytes, slots, rows}, strides[2] = {row_bytes, row_bytes * slots};
    const cuuint32_t box[3] = {(cuuint32_t)(row_bytes < 128 ? row_bytes : 128), kT, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               row_bytes < 128 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int D, int NQ, int MINB>
cudaError_t launch(const Q4AttnParams& pp, int batch, cudaStream_t st) {
    using L = Q4Layout<D>;
    Q4AttnParams p = pp;
    auto kernel = q4_attn_kernel<D, NQ, MINB>;
    static std::atomic<bool> configured[64];  // per device; the same value every time
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_relaxed);
    }
    constexpr int kOut = (kWarps / L::NG) * 8 * NQ * L::O_STRIDE * 4;  // epilogue's fp32 rows
    const int stage = (p.r.k_eq_v ? 1 : 2) * L::OP;
    int s = ((MINB >= 2 ? 100 : 200) * 1024 - 1024) / stage;
    s = s < 2 ? 2 : (s > kMaxStages ? kMaxStages : s);
    // no more stages than the chunk has tiles
    const int tiles = (p.r.max_seq_len < p.r.chunk ? p.r.max_seq_len : p.r.chunk) / kT + 2;
    if (s > tiles) s = tiles < 2 ? 2 : tiles;
    p.r.n_stages = s;
    const size_t smem = 1024 + (s * stage > kOut ? (size_t)s * stage : (size_t)kOut);
    const uint64_t slots = p.r.page_size ? p.r.page_size : p.r.cap;
    const uint64_t rows = (uint64_t)(p.r.page_size ? p.r.n_pages : batch) * p.r.n_kv;
    CUtensorMap km, vm;
    if (!encode_codes(&km, p.r.k, L::ROWB, slots, rows) ||
        !encode_codes(&vm, p.r.v, L::ROWB, slots, rows))
        return cudaErrorInvalidValue;
    const int rt = 8 * NQ, total = p.r.n_tok * p.r.G;
    const dim3 grid((unsigned)((total + rt - 1) / rt * p.r.n_split), p.r.n_kv, batch);
    cudaError_t e = launch_pdl(kernel, grid, dim3(kThreads), smem, st, km, vm, p);
    if (e == cudaSuccess && p.r.n_split > 1)
        e = launch_pdl(q4_merge_kernel<D>, dim3((unsigned)total, p.r.n_kv, batch),
                       dim3(kMergeThreads), 0, st, p.r, rt);
    return e;
}

}  // namespace

cudaError_t launch_q4_attn(const RowsParams& r, const Q4Cache& c, int head_dim, int batch,
                           cudaStream_t st) {
    const Q4AttnParams p{r, c.k_scales, c.v_codes ? c.v_scales : c.k_scales};
    const bool wide = q4_row_tile(r.n_tok * r.G) == 16;
    // two CTAs per SM where the query fragments leave registers for them
    switch (head_dim) {
        case 64: return wide ? launch<64, 2, 2>(p, batch, st) : launch<64, 1, 2>(p, batch, st);
        case 128: return wide ? launch<128, 2, 2>(p, batch, st) : launch<128, 1, 2>(p, batch, st);
        case 256: return wide ? launch<256, 2, 1>(p, batch, st) : launch<256, 1, 2>(p, batch, st);
        case 512: return wide ? launch<512, 2, 1>(p, batch, st) : launch<512, 1, 1>(p, batch, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gemma
