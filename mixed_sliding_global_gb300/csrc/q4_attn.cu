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
// A CTA takes 8 * NQ rows and a run of keys, 128 keys at a time: a unit's (sequence, KV head, row
// tile), a part of one that its cluster merges, or an equal share of the launch's. Ten warps: one thread of the first
// extra warp streams code tiles (TMA, 128-byte swizzle for rows of at least 128 bytes) and scales
// (bulk copies) into a ring of stages; the second extra warp describes the parts of units that the
// CTA will meet and turns their queries into fragments, one part ahead; eight warps each take 16
// keys of S over all of head_dim, exchange P through shared memory (one barrier per tile) and take a
// 64-column group of O (at head_dim < 512 the warps of a group share out the tile's keys). Two CTAs
// per SM (one at head_dim 512 with a V of its own, where two stages take 139 KB): 96 registers a thread, which the query fragments leave free up to head_dim 256 (8 rows) or
// 64 (16 rows); beyond they are read from shared memory for every tile.
// The softmax reference m is common to the CTA and lazy: a row's is 2^-6 of its largest weight when
// it is set, and moves only when a score exceeds it by more than 2^14, which the tile's one barrier
// votes on. P and its product with V's scale are rounded to fp16 (2^-11 each; the output is rounded
// to bf16, 2^-8); V's scales enter relative to the largest one of the chunk so far, scaled into
// [2^-1, 1), so that P and the product stay in fp16's normal range down to 2^-20 of the largest
// (below, a weight is off by 2^-31 of it: with m at the largest itself, it was 2^-25 from 2^-14 down).
// Everything else is fp32.
//
// What bounds it. Batch 64, lengths up to 16,385: the ring of 1,024 (16 / 8 heads, head_dim 256, 140
// MB): 45.8 us, 3.1 TB/s of the 6.8 that a copy reaches; the bf16 cache's kernel takes 88.7 for four
// times the bytes. The global layer (16 / 1, head_dim 512, K as V, 148 MB): 86 us, 1.7 TB/s, 200
// TFLOP/s; bf16 120. With the arithmetic left out the same loads take 34 and 51 us, without Q K^T
// 40 and 69, without P V 40 and 66: the unpacking (two integer instructions per pair of codes, and
// in P V a permutation per register that pairs keys; the integer pipe is 51% and 57% busy), the
// tensor pipe (20% and 39%) and their latencies with four warps per scheduler take turns rather
// than overlap (an instruction issues in half of the cycles). A tile of one CTA alone takes 0.6,
// 0.9, 1.25 and 2.6 us at head_dim 64 to 512 (8, 8, 8 and 16 rows), the launch 3.5 us besides.
// Tried and slower: multiplications for the rotations (ring 83 us against 76 then), one CTA per SM
// with deeper rings (51.6, 88.5), prefetches of later tiles into L2 (50), one box per tile at
// head_dim 512 (no change).
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
constexpr int kWarps = 8;           // consumer warps per CTA
constexpr int kThreads = (kWarps + 2) * 32;  // and two that load and prepare for them
constexpr int kMaxStages = 8;
constexpr float kTopLog2 = 6.f;    // a row's largest weight when its reference is set
constexpr float kLazyLog2 = 14.f;  // and the largest before it is set again
constexpr float kNoMax = -3.0e38f;  // reference before any key (finite: x - kNoMax is no NaN)
constexpr uint32_t kPairMask = 0x80078007u;

struct Q4AttnParams {
    RowsParams r;  // shapes, masks, q / out / partials (k, v: the code arrays)
    const __nv_bfloat16* k_scales;
    const __nv_bfloat16* v_scales;
    int batch;
    int balanced;     // equal shares of the launch's key tiles per CTA (else whole units)
    int cluster;      // CTAs that share a unit's tiles, a cluster (1 with equal shares)
    int2* info;       // [units]: {first part row tile, last CTA} of a shared unit, or {-1, -1}
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
// Loads from shared memory at 32-bit addresses (generic pointers would cost the tile loop a pair of
// registers each, and this kernel has none to spare).
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t v, uint32_t w) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(v), "r"(w) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((uint16_t)v) : "memory");
}

// Slot j of a word: its pair of codes as two fp16 numbers code * 2^-24.
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int j) {
    return __funnelshift_r(word, word, 4 * j) & kPairMask;
}

// Barriers of the consumer warps; the vote also ORs a flag over their threads.
__device__ __forceinline__ void consumer_sync() { named_bar_sync(1, kWarps * 32); }
__device__ __forceinline__ bool consumer_vote(bool flag) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)flag), "n"(kWarps * 32)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ uint32_t peer_addr(const void* local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(r)
                 : "r"(smem_u32(local)), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// Barrier of the cluster's threads that still run, ordering their shared memory.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

template <int D>
struct Q4Layout {
    static constexpr int NG = D / kQ4Group;                     // scale groups per row
    static constexpr int ROWB = D / 2;                          // code bytes per row
    static constexpr int BOXB = ROWB < 128 ? ROWB : 128;        // bytes per row of one TMA box
    static constexpr int CODES = kT * ROWB;                     // one tile of codes
    static constexpr int SCALES = kT * NG * 2;                  // and of scales
    static constexpr int OP = CODES + (SCALES + 1023) / 1024 * 1024;  // one operand of a stage
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

// Rounded-down first position of a step's keys (from the first query's window): 32 keeps scale
// rows 16-byte aligned; a tile must not wrap round a ring or leave a page.
__device__ __forceinline__ int first_key(const RowsParams& p, int len) {
    const int lo = p.is_sliding ? max(0, len - p.n_tok - p.window + 1) : 0;
    return lo & ~((p.ring || p.page_size ? kT : 32) - 1);
}
__device__ __forceinline__ bool bad_length(const RowsParams& p, int len) {
    return len < p.n_tok || (!p.ring && len > p.cap) || len > p.max_seq_len;
}
// Key tiles of a unit (KV head, row tile) of a sequence; an invalid sequence has one, whose CTA
// writes the zeros.
__device__ __forceinline__ int unit_tiles(const RowsParams& p, int len) {
    return bad_length(p, len) ? 1 : (len - first_key(p, len) + kT - 1) / kT;
}

// The work of a launch is one line of places: sequences in order, a sequence's units in order, a
// unit's tiles in order behind kHead empty places (a part's set-up and its rows cost about that
// many tiles). CTA c of C takes places [c total / C, (c + 1) total / C), so every CTA has about
// the same work whatever the lengths; it meets whole units and at most two parts of units, which
// the merge launch puts together. Where a place x lies:
constexpr int kHead = 1;
__device__ __forceinline__ long long share_start(long long total, int C, int c) {
    return total * c / C;
}
__device__ __forceinline__ int share_of(long long total, int C, long long x) {
    return (int)(((x + 1) * C + total - 1) / total) - 1;
}

// First of n tiles that CTA `rank` of c takes of a unit (rank c: n).
__device__ __forceinline__ int cluster_start(int n, int c, int rank) {
    return (int)((long long)n * rank / c);
}

// Sum over the CTA's threads of their values before this one, and the total.
__device__ __forceinline__ int cta_scan(int v, int* s_warp, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    __syncthreads();
    return before + x - v;
}

// One part of a unit: sequence b, KV head kvh, row tile rt, key tiles [t0, t1) of n.
struct Part {
    int b, kvh, rt, t0, t1, n, len;
};
struct Walk {
    int b, u, t, n, len;  // next place: tile t (before 0: the head) of unit u of sequence b
    __device__ void enter(const RowsParams& p, int seq) {
        b = seq;
        len = p.seq_lens[seq];
        n = unit_tiles(p, len);
    }
    // The part of the current unit within the next `left` places (possibly without tiles), and
    // step on; left becomes what is left behind it.
    __device__ Part take(const RowsParams& p, int n_rt, int upb, int batch, int& left) {
        const int to = n - t < left ? n : t + left;
        left -= to - t;
        const Part s{b, u / n_rt, u % n_rt, max(t, 0), to, n, len};
        t = to;
        if (t == n) {
            t = -kHead;
            if (++u == upb) {
                u = 0;
                if (b + 1 < batch) enter(p, b + 1);
            }
        }
        return s;
    }
};

// What the consumer warps need of the current part (in shared memory: it would take a dozen
// registers of every thread through the tile loop).
struct Job {
    Part part;
    int last;  // no part: the share ends
    int row0, n_rows, key_first, whole, slot;
    int lo_all, ke;      // keys of any row
    int lo_max, hi_min;  // keys that every row of the tile may see
};

// A unit's rows from its cluster of c CTAs (of n tiles in all; a CTA without tiles has no part), the
// rows in `rows` and their m and l in `ml_rows` of each, through distributed shared memory:
// M = max m_k, out = sum 2^(m_k - M) O_k / sum 2^(m_k - M) l_k, 16 bytes of O per thread at a time.
// out: row R = row0 + r of a KV head lies (R / G * n_q + R % G) * D behind it.
template <int D>
__device__ __forceinline__ void cluster_merge(const uint8_t* rows, const float2* ml_rows, int c, int n,
                                           int row0, int n_rows, int G, int n_q,
                                           __nv_bfloat16* out) {
    cluster_barrier();
    for (int i = blockIdx.x % c * (kWarps * 32) + threadIdx.x; i < n_rows * (D / 4);
         i += c * (kWarps * 32)) {
        const int r = i / (D / 4), x = i - r * (D / 4);
        float2 ml[kQ4MaxCluster];
        float4 v[kQ4MaxCluster];
        float M = kNoMax;
#pragma unroll
        for (int k = 0; k < kQ4MaxCluster; ++k) {
            ml[k] = make_float2(kNoMax, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < c && cluster_start(n, c, k + 1) > cluster_start(n, c, k)) {
                ml[k] = ld_peer2(peer_addr(&ml_rows[r], k));
                v[k] = ld_peer4(peer_addr(rows, k) + (r * D + x * 4) * 4);
            }
        }
#pragma unroll
        for (int k = 0; k < kQ4MaxCluster; ++k) M = fmaxf(M, ml[k].x);
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kQ4MaxCluster; ++k) {
            const float w = exp2f(ml[k].x - M);
            l = fmaf(w, ml[k].y, l);
            acc.x = fmaf(w, v[k].x, acc.x);
            acc.y = fmaf(w, v[k].y, acc.y);
            acc.z = fmaf(w, v[k].z, acc.z);
            acc.w = fmaf(w, v[k].w, acc.w);
        }
        const float il = 1.f / l;
        const int R = row0 + r, tok = R / G;
        *reinterpret_cast<uint2*>(out + ((size_t)tok * n_q + R - tok * G) * D + x * 4) =
            make_uint2(pack_bf16(acc.x * il, acc.y * il), pack_bf16(acc.z * il, acc.w * il));
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
}

// PAIR: at most four rows (NQ = 1; the ring above 46.2 us against 52.3 with eight columns of rows,
// one unit of 4 rows 9.1 against 9.3). P V then takes the pair of codes of a word's slot as two
// operand elements of one key, weighted (P, 0) in columns 0..3 and (0, P) in columns 4..7: the
// even and the odd output columns come out side by side and no codes are re-paired across keys.
// CLUSTER: several CTAs share a unit (an instantiation of its own: the tile loop's registers would
// pay for the merge).
template <int D, int NQ, bool PAIR, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, kQ4CtasPerSm)
    q4_attn_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ Q4AttnParams pp) {
    pdl_launch_dependents();
    using L = Q4Layout<D>;
    constexpr int RT = 8 * NQ;
    constexpr int NG = L::NG;
    constexpr int KSP = kWarps / NG;        // warps that share a column group
    constexpr int KW = kT / KSP;            // keys per warp of a tile in P V
    // query fragments in registers where they leave room for the rest (else in shared memory)
    constexpr bool QREG = NQ == 1 ? D <= 256 : D <= 64;
    constexpr int PW = PAIR ? 16 : 8 * NQ;  // halves of P per key
    constexpr bool QPRE = NQ == 1;          // the producer prepares the next part's query rows
    const RowsParams& p = pp.r;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ __align__(16) __half sP[2][kT * PW];
    __shared__ __align__(16) __half sV[kWarps][PAIR ? 2 * KW : KW];
    __shared__ __align__(16) uint32_t sQ[QPRE ? 2 : 1][D / 16][32][2 * NQ];
    __shared__ float sMax[kWarps][RT], sSum[kWarps][RT];
    __shared__ __align__(8) float sInv[2][RT];
    __shared__ __align__(8) float2 sMl[CLUSTER ? RT : 1];  // of a part for its cluster: the rows' m and l
    __shared__ int sScan[kThreads / 32], sAt[3];
    // the part being worked on and the one that the producer prepares
    __shared__ Job sJob[2];
    __shared__ __align__(8) uint64_t job_full[2], job_empty[2];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tq = lane & 3;
    const int nops = p.k_eq_v ? 1 : 2;
    const int stage_bytes = nops * L::OP;
    const int S = p.n_stages;
    float* sO = reinterpret_cast<float*>(smem + S * stage_bytes);  // [KSP - 1][RT][D]
    const int rows_total = p.n_tok * p.G;
    const int n_rt = (rows_total + RT - 1) / RT, upb = n_rt * p.n_kv;
    const int batch = pp.batch;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(&job_full[j], 1);
            mbar_init(&job_empty[j], kWarps);
        }
        fence_barrier_init();
    }
    pdl_wait();
    // where this CTA's share starts
    Walk walk;
    int left;                   // places of this CTA
    long long all = 0, x0 = 0;  // places of the launch, first one of this CTA
    int C = 0;                  // CTAs with a share (no more than places)
    if (!CLUSTER && pp.balanced) {
        const int per = (batch + kThreads - 1) / kThreads, b0 = min((int)threadIdx.x * per, batch);
        const int b1 = min(b0 + per, batch);
        int mine = 0, total;
        for (int b = b0; b < b1; ++b) mine += unit_tiles(p, p.seq_lens[b]) + kHead;
        const int before = cta_scan(mine, sScan, total);
        all = (long long)total * upb;
        C = all < gridDim.x ? (int)all : (int)gridDim.x;
        if ((int)blockIdx.x >= C) return;
        x0 = share_start(all, C, blockIdx.x);
        left = (int)(share_start(all, C, blockIdx.x + 1) - x0);
        if (x0 >= (long long)before * upb && x0 < (long long)(before + mine) * upb) {
            long long x = x0 - (long long)before * upb;
            int b = b0, n = unit_tiles(p, p.seq_lens[b]) + kHead;
            while (x >= (long long)n * upb) {
                x -= (long long)n * upb;
                n = unit_tiles(p, p.seq_lens[++b]) + kHead;
            }
            sAt[0] = b;
            sAt[1] = (int)(x / n);
            sAt[2] = (int)(x % n) - kHead;
        }
        __syncthreads();
        walk.enter(p, sAt[0]);
        walk.u = sAt[1];
        walk.t = sAt[2];
    } else {  // a cluster per unit
        const int c = CLUSTER ? pp.cluster : 1;
        const int unit = blockIdx.x / c, rank = blockIdx.x - unit * c;
        walk.enter(p, unit / upb);
        walk.u = unit % upb;
        walk.t = rank ? cluster_start(walk.n, c, rank) : -kHead;
        left = (CLUSTER ? cluster_start(walk.n, c, rank + 1) : walk.n) - walk.t;
        __syncthreads();
    }

    // Element offset in q and out of row r of a part's tile: token (row0 + r) / G, head
    // kvh * G + (row0 + r) % G.
    auto row_at = [&](const Job& j, int r) {
        const int R = j.row0 + r, tok = R / p.G;
        return (((size_t)j.part.b * p.n_tok + tok) * p.n_q + j.part.kvh * p.G + (R - tok * p.G)) *
               (size_t)D;
    };
    // One warp turns query row r of a part into fp16 fragments: lane (g, tq) will hold, of row g of
    // each 8-row tile, elements 16 tq .. 16 tq + 15 of every group, the ones whose codes it reads.
    // The row is scaled by a power of two that brings its largest element into [2^13, 2^14)
    // (exact unless an element is below 2^-30 of that, then off by at most 2^-38 of it: 2^-25, half of
    // fp16's smallest step).
    auto prepare_row = [&](const Job& j, int slot, int r) {
        constexpr int CH = (D / 8 + 31) / 32;
        uint4 raw[CH];
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = c * 32 + lane;
            raw[c] = make_uint4(0u, 0u, 0u, 0u);
            if (r < j.n_rows && ch < D / 8)
                raw[c] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                        row_at(j, r))[ch];
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        }
        mx = __reduce_max_sync(0xffffffffu, mx);
        // biased exponent of the largest element -> factor 2^(13 - (exponent - 127))
        const float f =
            __uint_as_float((uint32_t)(267 - min(max((int)(mx >> 7), 13), 254)) << 23);
        // a score is the sum of products times this times 2^12 (the codes' 2^24 in two halves: with
        // all of it on one side the keys' or the queries' large numbers would leave fp32's range)
        if (lane == 0)
            sInv[slot][r] = (p.softcap > 0.f ? p.cap_inner : p.scale_log2) * 4096.f / f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = c * 32 + lane;  // elements 8 ch .. 8 ch + 7
            if (ch >= D / 8) continue;
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[k] = pack_f16(__uint_as_float(w[k] << 16) * f,
                                __uint_as_float(w[k] & 0xffff0000u) * f);
            const int ks = (ch >> 3) * 4 + 2 * (ch & 1), ln = (r & 7) * 4 + ((ch >> 1) & 3);
            auto& q = sQ[QPRE ? slot : 0];
            *reinterpret_cast<uint2*>(&q[ks][ln][(r >> 3) * 2]) = make_uint2(h[0], h[1]);
            *reinterpret_cast<uint2*>(&q[ks + 1][ln][(r >> 3) * 2]) = make_uint2(h[2], h[3]);
        }
    };

    if (warp == kWarps) {
        // the share's tiles in order, one thread issuing the copies
        if (lane == 0) {
            const int slots = kv_row_slots(p);
            int s = 0, round = 0;  // stage, and how often the ring went round
            while (left > 0) {
                const Part part = walk.take(p, n_rt, upb, batch, left);
                const bool bad = bad_length(p, part.len);
                const int key_first = first_key(p, part.len);
                for (int t = part.t0; t < part.t1; ++t) {
                    uint64_t* bar = &full[s];
                    uint8_t* st = smem + s * stage_bytes;
                    if (round > 0 && !mbar_wait(&empty[s], (round - 1) & 1, p.err)) {
                        left = 0;
                        break;
                    }
                    if (++s == S) {
                        s = 0;
                        ++round;
                    }
                    if (bad) {  // no keys: the stage is passed on empty
                        mbar_arrive(bar);
                        continue;
                    }
                    int row = 0, slot = 0;
                    const bool ok = kv_place(p, part.b, part.kvh, key_first + t * kT, row, slot);
                    // scale rows that exist (a tile may reach behind the last slot; capacities
                    // and tile starts are multiples of 32, so the copies stay multiples of 16 B)
                    const uint32_t sbytes = ok ? (uint32_t)(min(kT, slots - slot) * NG * 2) : 0u;
                    if (!ok) {  // a bad page reads as zeros
                        report(p.err, GEMMA_DEVERR_PAGE);
                        row = p.n_pages * p.n_kv;
                        for (int o = 0; o < nops; ++o)
                            for (int k = 0; k < L::SCALES / 16; ++k)
                                reinterpret_cast<uint4*>(st + o * L::OP + L::CODES)[k] =
                                    make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();  // (a later copy into the stage comes behind them)
                    }
                    mbar_arrive_expect_tx(bar, (uint32_t)nops * (L::CODES + sbytes));
                    for (int o = 0; o < nops; ++o) {
                        uint8_t* dst = st + o * L::OP;
#pragma unroll
                        for (int c = 0; c < L::ROWB / L::BOXB; ++c)
                            tma_load_3d(dst + c * kT * 128, o ? &vmap : &kmap, c * 128, slot, row,
                                        bar);
                        if (sbytes)
                            bulk_g2s(dst + L::CODES,
                                     (o ? pp.v_scales : pp.k_scales) +
                                         ((size_t)row * slots + slot) * NG,
                                     sbytes, bar);
                    }
                }
            }
            // no copy outlives the CTA, whatever the consumers waited for
            for (int i = 0; i < S; ++i) {
                const int uses = round + (i < s ? 1 : 0);
                if (uses > 0) mbar_wait(&full[i], (uses - 1) & 1, p.err);
            }
        }
        return;
    }
    if (warp == kWarps + 1) {
        // The share's parts: their descriptions and, for up to eight rows, their query fragments,
        // one part ahead of the consumers.
        int n_job = 0;
        for (long long x = x0; left > 0;) {
            const int js = n_job & 1, before = left;
            Job j;
            j.part = walk.take(p, n_rt, upb, batch, left);
            const Part& part = j.part;
            const long long first = x + (before - left) - part.t1;  // place of the unit's tile 0
            x += before - left;
            if (part.t1 <= part.t0) continue;  // a head only
            j.last = 0;
            j.row0 = part.rt * RT;
            j.n_rows = min(RT, rows_total - j.row0);
            j.whole = part.t0 == 0 && part.t1 == part.n;
            j.slot = 2 * (int)blockIdx.x + (n_job > 0);
            j.key_first = first_key(p, part.len);
            j.lo_all = p.is_sliding ? max(0, part.len - p.n_tok - p.window + 1) : 0;
            j.ke = min(part.len, j.key_first + part.t1 * kT);
            const int pos0 = part.len - p.n_tok + j.row0 / p.G;
            const int pos1 = part.len - p.n_tok + (j.row0 + j.n_rows - 1) / p.G;
            j.lo_max = p.is_sliding ? max(0, pos1 - p.window + 1) : 0;
            j.hi_min = min(pos0 + 1, j.ke);
            if (n_job >= 2 && !mbar_wait(&job_empty[js], (n_job / 2 - 1) & 1, p.err)) return;
            if (lane == 0) {
                sJob[js] = j;
                if (!CLUSTER && pp.balanced && part.t0 == 0)  // who shares the unit, for the merge
                    pp.info[(part.b * p.n_kv + part.kvh) * n_rt + part.rt] =
                        j.whole ? make_int2(-1, -1)
                                : make_int2(j.slot, share_of(all, C, first + part.n - 1));
            }
            // (the consumers prepare the first part's rows themselves, one warp each)
            if (QPRE && n_job > 0 && !bad_length(p, part.len)) {
#pragma unroll (PAIR ? 4 : 2)
                for (int r = 0; r < RT; ++r)
                    if (r < j.n_rows || n_job == 1) prepare_row(j, js, r);  // (the rest stay zero)
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&job_full[js]);
            ++n_job;
        }
        // the end of the share
        const int js = n_job & 1;
        if (n_job >= 2 && !mbar_wait(&job_empty[js], (n_job / 2 - 1) & 1, p.err)) return;
        if (lane == 0) {
            sJob[js].last = 1;
            mbar_arrive(&job_full[js]);
        }
        return;
    }

    const int wg = warp % NG, ksp = warp / NG;
    const uint32_t smem0 = smem_u32(smem), aV = smem_u32(sV[warp]);
    const int krow = warp * 16 + key_of_row<D>(g);  // this lane's keys of S: krow, krow + 8
    // byte offsets in a tile of the words this lane reads: for S, key krow (krow + 8 lies 8 rows
    // on), group i at sOff[i % 4] in box i / 4; for P V, an even and an odd key of its group's words
    constexpr int XO = L::BOXB < 128 ? 1 : (NG < 4 ? NG : 4);
    int sOff[XO], vOff[2];
#pragma unroll
    for (int i = 0; i < XO; ++i) sOff[i] = code_off<D>(krow, i * 32 + tq * 8);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        vOff[i] = code_off<D>(ksp * KW + 2 * tq + i, wg * 32 + g * 4);
    const int vsOff = L::CODES + ((ksp * KW + lane) * NG + wg) * 2;  // V's scale of key lane
    auto s_off = [&](int i) {
        return L::BOXB < 128 ? sOff[0] + i * 32 : sOff[i % XO] + (i / 4) * (kT * 128);
    };
    int done = 0, s = 0;    // tiles taken, the next one's stage
    uint32_t phase = 0;     // and the parity of its barrier
    auto next_stage = [&]() {
        ++done;
        if (++s == S) {
            s = 0;
            phase ^= 1;
        }
    };
    bool ok = true;
    for (int n_job = 0;; ++n_job) {
        const int js = n_job & 1;
        // (the vote lets every warp leave together if one gave up waiting)
        if (consumer_vote(!mbar_wait(&job_full[js], (n_job >> 1) & 1, p.err))) break;
        const Job& job = sJob[js];
        if (job.last) break;
        if (bad_length(p, job.part.len)) {
            // (its stage holds nothing, but counts: consumers that ran past stages not yet given would
            // take a phase of the ring for another)
            if (ok) ok = mbar_wait(&full[s], phase, p.err);
            if (threadIdx.x == 0) report(p.err, GEMMA_DEVERR_SEQ_LEN);
            for (int i = threadIdx.x; i < job.n_rows * (D / 8); i += kWarps * 32)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                          row_at(job, i / (D / 8)) + i % (D / 8) * 8) =
                    make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&empty[s]);
                mbar_arrive(&job_empty[js]);
            }
            next_stage();
            continue;
        }
        if (!QPRE || n_job == 0) {
            for (int r = warp; r < RT; r += kWarps) prepare_row(job, js, r);
            consumer_sync();
        }
        uint32_t qf[QREG ? D / 16 : 1][NQ][2];
        if (QREG) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    qf[QREG ? k : 0][n][0] = sQ[QPRE ? js : 0][k][lane][2 * n];
                    qf[QREG ? k : 0][n][1] = sQ[QPRE ? js : 0][k][lane][2 * n + 1];
                }
        }
        // the rows whose scores this lane holds: 8 n + 2 tq + c
        float m_run[NQ][2], l_run[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m_run[n][c] = kNoMax;
                l_run[n][c] = 0.f;
            }
        float o[4][NQ][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NQ; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        int v_exp = 6;  // biased exponent that V's scales are relative to

        const uint32_t tQ = smem_u32(sQ[QPRE ? js : 0][0][lane]);
        for (int t = job.part.t0, t1 = job.part.t1; t < t1; ++t) {
            if (ok) ok = mbar_wait(&full[s], phase, p.err);
            const uint32_t tK = smem0 + s * stage_bytes;
            const uint32_t tV = tK + (nops - 1) * L::OP;
            const int key0 = job.key_first + t * kT;

            // (1) S of 16 keys
            float sv[NQ][4];
#pragma unroll
            for (int n = 0; n < NQ; ++n) sv[n][0] = sv[n][1] = sv[n][2] = sv[n][3] = 0.f;
            {
                alignas(16) uint32_t ska[(NG + 1) / 2], skb[(NG + 1) / 2];  // scales of the two keys, bf16 pairs
                const uint32_t sk = tK + L::CODES + krow * (NG * 2);
                if (NG == 8) {
                    const uint4 a = lds128(sk), b = lds128(sk + 8 * NG * 2);
                    *reinterpret_cast<uint4*>(ska) = a;
                    *reinterpret_cast<uint4*>(skb) = b;
                } else if (NG == 4) {
                    const uint2 a = lds64(sk), b = lds64(sk + 8 * NG * 2);
                    *reinterpret_cast<uint2*>(ska) = a;
                    *reinterpret_cast<uint2*>(skb) = b;
                } else if (NG == 2) {
                    ska[0] = lds32(sk);
                    skb[0] = lds32(sk + 8 * NG * 2);
                } else {
                    ska[0] = lds16(sk);
                    skb[0] = lds16(sk + 8 * NG * 2);
                }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const uint2 wa = lds64(tK + s_off(i)), wb = lds64(tK + s_off(i) + 8 * L::BOXB);
                    float acc[NQ][4];
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint32_t xa = ks < 2 ? wa.x : wa.y, xb = ks < 2 ? wb.x : wb.y;
                        const int j = 2 * (ks & 1);
                        const uint32_t a0 = code_pair(xa, j), a1 = code_pair(xb, j);
                        const uint32_t a2 = code_pair(xa, j + 1), a3 = code_pair(xb, j + 1);
                        alignas(16) uint32_t bq[2 * NQ];
                        if (QREG) {
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                bq[2 * n] = qf[QREG ? i * 4 + ks : 0][n][0];
                                bq[2 * n + 1] = qf[QREG ? i * 4 + ks : 0][n][1];
                            }
                        } else if (NQ == 2) {
                            const uint4 v = lds128(tQ + (i * 4 + ks) * (32 * 8 * NQ));
                            *reinterpret_cast<uint4*>(bq) = v;
                        } else {
                            const uint2 v = lds64(tQ + (i * 4 + ks) * (32 * 8 * NQ));
                            *reinterpret_cast<uint2*>(bq) = v;
                        }
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            if (ks == 0) mma_f16_zero(acc[n], a0, a1, a2, a3, bq[2 * n], bq[2 * n + 1]);
                            else mma_f16(acc[n], a0, a1, a2, a3, bq[2 * n], bq[2 * n + 1]);
                        }
                    }
                    const float fa = __uint_as_float(i & 1 ? ska[i / 2] & 0xffff0000u : ska[i / 2] << 16);
                    const float fb = __uint_as_float(i & 1 ? skb[i / 2] & 0xffff0000u : skb[i / 2] << 16);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        sv[n][0] = fmaf(acc[n][0], fa, sv[n][0]);
                        sv[n][1] = fmaf(acc[n][1], fa, sv[n][1]);
                        sv[n][2] = fmaf(acc[n][2], fb, sv[n][2]);
                        sv[n][3] = fmaf(acc[n][3], fb, sv[n][3]);
                    }
                }
            }
            // scores in log2 units; masked keys -inf (a tile inside every row's range has none)
            const bool edge = key0 < job.lo_max || key0 + kT > job.hi_min;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float2 inv = *reinterpret_cast<const float2*>(&sInv[js][n * 8 + 2 * tq]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sv[n][k] = sv[n][k] * (k & 1 ? inv.y : inv.x) * 4096.f;
            }
            if (p.softcap > 0.f) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sv[n][k] = p.cap_log2 * tanhf(sv[n][k]);
            }
            if (edge) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = min(n * 8 + 2 * tq + c, job.n_rows - 1);
                        const int pos = job.part.len - p.n_tok + (job.row0 + r) / p.G;
                        const int lo = p.is_sliding ? pos - p.window + 1 : 0;
                        const int hi = min(pos + 1, job.ke);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = key0 + krow + 8 * h;
                            if (key < lo || key >= hi) sv[n][2 * h + c] = -INFINITY;
                        }
                    }
            }
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    grow = grow || fmaxf(sv[n][c], sv[n][c + 2]) > m_run[n][c] + kLazyLog2;
            const uint32_t P = smem_u32(sP[done & 1]);
            float l_tile[NQ][2];
            auto exponentiate = [&]() {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    float pr[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) pr[k] = fast_exp2(sv[n][k] - m_run[n][k & 1]);
                    l_tile[n][0] = pr[0] + pr[2];
                    l_tile[n][1] = pr[1] + pr[3];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = krow + 8 * h;
                        if (PAIR) {  // [key][8] words: columns q (P, 0), 4 + q (0, P)
                            if (tq < 2) {
                                const uint32_t d = P + key * 32 + 8 * tq;
                                const uint32_t e = pack_f16(pr[2 * h], 0.f);
                                const uint32_t f = pack_f16(pr[2 * h + 1], 0.f);
                                sts64(d, e, f);
                                sts64(d + 16, e << 16, f << 16);
                            }
                        } else {     // planes of 8 rows
                            sts32(P + (n * kT + key) * 16 + 4 * tq,
                                  pack_f16(pr[2 * h], pr[2 * h + 1]));
                        }
                    }
                }
            };
            exponentiate();
            // V's scales of this warp's keys and group, as fp16 relative to 2^v_exp
            {
                uint32_t sb[(KW + 31) / 32], mx = 0;
#pragma unroll
                for (int i = 0; i < (KW + 31) / 32; ++i) {
                    const int k = i * 32 + lane, key = key0 + ksp * KW + k;
                    sb[i] = k < KW ? lds16(tV + vsOff + i * 64 * NG) : 0;
                    if (edge && (key < job.lo_all || key >= job.ke)) sb[i] = 0;  // may hold anything
                    mx = max(mx, sb[i]);
                }
                // (a NaN scale, exponent 255, leaves NaN in its column group either way; 252 is a scale's largest)
                mx = min(__reduce_max_sync(0xffffffffu, mx) >> 7, 252u);
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
                const float f = __uint_as_float((uint32_t)(253 - v_exp) << 23);  // 2^(-1-(v_exp-127))
#pragma unroll
                for (int i = 0; i < (KW + 31) / 32; ++i)
                    if (i * 32 + lane < KW) {
                        const float x = __uint_as_float(sb[i] << 16) * f;
                        if (PAIR)
                            sts32(aV + (i * 32 + lane) * 4, pack_f16(x, x));
                        else
                            sts16(aV + (i * 32 + lane) * 2, pack_f16(x, 0.f));
                    }
            }
            if (consumer_vote(grow)) {
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
                consumer_sync();
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = m_run[n][c];
#pragma unroll
                        for (int w = 0; w < kWarps; ++w)
                            mx = fmaxf(mx, sMax[w][n * 8 + 2 * tq + c] - kTopLog2);
                        float a = 1.f;
                        if (mx > m_run[n][c]) {
                            a = fast_exp2(m_run[n][c] - mx);  // 0 from kNoMax
                            m_run[n][c] = mx;
                            l_run[n][c] *= a;
                        }
                        if (PAIR) a = __shfl_sync(0xffffffffu, a, (lane & ~3) | (tq & 1));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[i][n][c] *= a;
                            o[i][n][c + 2] *= a;
                        }
                    }
                exponentiate();
                consumer_sync();
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) l_run[n][c] += l_tile[n][c];

            // (2) O of 64 columns over this warp's keys
            if constexpr (PAIR) {
                // 8 keys per step: operand elements 2 tq, 2 tq + 1 are the codes of key 2 tq's
                // slot pair, 2 tq + 8, 2 tq + 9 those of key 2 tq + 1; MMA rows g, g + 8 of tile i
                // are columns (8 g + 4 i, + 1) and (8 g + 4 i + 2, + 3) of the group
#pragma unroll
                for (int kk = 0; kk < KW; kk += 8) {
                    const int kt = ksp * KW + kk + 2 * tq;
                    const uint2 sc = lds64(aV + (kk + 2 * tq) * 4);
                    const uint32_t b0 = mul_f16x2(lds32(P + kt * 32 + g * 4), sc.x);
                    const uint32_t b1 = mul_f16x2(lds32(P + kt * 32 + 32 + g * 4), sc.y);
                    const uint32_t w0 = lds32(tV + vOff[0] + kk * L::BOXB);
                    const uint32_t w1 = lds32(tV + vOff[1] + kk * L::BOXB);
                    mma_f16(o[0][0], code_pair(w0, 0), code_pair(w0, 1),
                            code_pair(w1, 0), code_pair(w1, 1), b0, b1);
                    mma_f16(o[1][0], code_pair(w0, 2), code_pair(w0, 3),
                            code_pair(w1, 2), code_pair(w1, 3), b0, b1);
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < KW; kk += 16) {
                    const int kt = ksp * KW + kk;
                    uint32_t bf[NQ][2];
                    if (NQ == 2) {
                        const uint32_t a = P + ((lane >> 4) * kT + kt + (lane & 15)) * 16;
                        ldsm_x4_t(a, bf[0][0], bf[0][1], bf[NQ - 1][0], bf[NQ - 1][1]);
                    } else {
                        const uint32_t a = P + (kt + (lane & 15)) * 16;
                        asm volatile(
                            "ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                            : "=r"(bf[0][0]), "=r"(bf[0][1])
                            : "r"(a));
                    }
                    const uint32_t s0 = lds32(aV + (kk + 2 * tq) * 2);
                    const uint32_t s1 = lds32(aV + (kk + 2 * tq + 8) * 2);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        bf[n][0] = mul_f16x2(bf[n][0], s0);
                        bf[n][1] = mul_f16x2(bf[n][1], s1);
                    }
                    uint32_t w[4];  // words of keys 2 tq, + 1, + 8, + 9: columns 8 g .. 8 g + 7
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = lds32(tV + vOff[k & 1] + (kk + 8 * (k >> 1)) * L::BOXB);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // MMA rows g, g + 8: columns 8 g + 2 i, + 1
                        uint32_t r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) r[k] = code_pair(w[k], i);
                        const uint32_t a0 = __byte_perm(r[0], r[1], 0x5410);
                        const uint32_t a1 = __byte_perm(r[0], r[1], 0x7632);
                        const uint32_t a2 = __byte_perm(r[2], r[3], 0x5410);
                        const uint32_t a3 = __byte_perm(r[2], r[3], 0x7632);
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
                            mma_f16(o[i][n], a0, a1, a2, a3, bf[n][0], bf[n][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            next_stage();
        }

        // ---------------------------------- the part's rows ----------------------------------
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = l_run[n][c];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
                if (g == 0) sSum[warp][n * 8 + 2 * tq + c] = l * 0.015625f;  // 2^-kTopLog2
            }
        // this lane's columns of rows q(n, c): x = wg * 64 + 8 g .. + 7
        // (2^(v_exp - 127 + 1), and 2^-6 as for l: a largest weight of one keeps V's range)
        const float f2 = __uint_as_float((uint32_t)(v_exp - 5) << 23);
        float v[NQ][2][8];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (PAIR) {
                        // lanes tq < 2 hold the even columns of rows 2 tq + c, tq >= 2 the odd ones
                        // of rows 2 (tq - 2) + c; o[i / 2]: columns 8 g + 4 (i / 2) + 2 (i & 1)
                        const float mine = o[i / 2][0][c + 2 * (i & 1)] * 16777216.f * f2;
                        const float other = __shfl_xor_sync(0xffffffffu, mine, 2);
                        v[n][c][2 * i] = tq < 2 ? mine : other;
                        v[n][c][2 * i + 1] = tq < 2 ? other : mine;
                    } else {
                        v[n][c][2 * i] = o[i][n][c] * 16777216.f * f2;
                        v[n][c][2 * i + 1] = o[i][n][c + 2] * 16777216.f * f2;
                    }
                }
        if (KSP > 1 && ksp > 0 && (!PAIR || tq < 2)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float4* d = reinterpret_cast<float4*>(
                        sO + ((size_t)(ksp - 1) * RT + n * 8 + 2 * tq + c) * D + wg * 64 + g * 8);
                    d[0] = make_float4(v[n][c][0], v[n][c][1], v[n][c][2], v[n][c][3]);
                    d[1] = make_float4(v[n][c][4], v[n][c][5], v[n][c][6], v[n][c][7]);
                }
        }
        consumer_sync();
        if (ksp == 0 && (!PAIR || tq < 2)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = n * 8 + 2 * tq + c, x = wg * 64 + g * 8;
                    if (r >= job.n_rows) continue;
#pragma unroll
                    for (int h = 1; h < KSP; ++h)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[n][c][k] += sO[((size_t)(h - 1) * RT + r) * D + x + k];
                    float l = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) l += sSum[w][r];
                    const float* y = v[n][c];
                    if (job.whole) {
                        const float il = 1.f / l;
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row_at(job, r) + x) =
                            make_uint4(pack_bf16(y[0] * il, y[1] * il), pack_bf16(y[2] * il, y[3] * il),
                                       pack_bf16(y[4] * il, y[5] * il), pack_bf16(y[6] * il, y[7] * il));
                    } else if (CLUSTER) {  // (the stages are done with)
                        float4* d = reinterpret_cast<float4*>(smem) + (r * D + x) / 4;
                        d[0] = make_float4(y[0], y[1], y[2], y[3]);
                        d[1] = make_float4(y[4], y[5], y[6], y[7]);
                        if (wg == 0 && g == 0) sMl[CLUSTER ? r : 0] = make_float2(m_run[n][c], l);
                    } else {
                        const size_t pr = (size_t)job.slot * RT + r;
                        float4* d = reinterpret_cast<float4*>(p.o_part + pr * D + x);
                        d[0] = make_float4(y[0], y[1], y[2], y[3]);
                        d[1] = make_float4(y[4], y[5], y[6], y[7]);
                        if (wg == 0 && g == 0)
                            reinterpret_cast<float2*>(p.ml_part)[pr] = make_float2(m_run[n][c], l);
                    }
                }
        }
        // sSum and sO are rewritten only behind another part's votes; the job's slot is free
        __syncwarp();
        if (lane == 0) mbar_arrive(&job_empty[js]);
    }
    if (!CLUSTER) return;

    const int unit = blockIdx.x / pp.cluster, b = unit / upb, u = unit - b * upb;
    const int row0 = u % n_rt * RT, n = unit_tiles(p, p.seq_lens[b]);
    // (one tile, or a bad length: one CTA wrote the rows)
    cluster_merge<D>(smem, sMl, pp.cluster, n, row0, n > 1 ? min(RT, rows_total - row0) : 0, p.G,
                     p.n_q,
                     static_cast<__nv_bfloat16*>(p.out) +
                         ((size_t)b * p.n_tok * p.n_q + u / n_rt * p.G) * D);
}

// Merge of the rows of units that several CTAs shared: M = max m_c,
// out = sum 2^(m_c - M) O_c / sum 2^(m_c - M) l_c. A CTA takes `cols` columns of one row: all of
// them, or 64 when there are few rows (a long cache of one sequence leaves a part per SM, and many
// short loads at once hide their latency): with 16 rows of 8192 keys the step takes 13.6 us by 64
// columns and 21.8 by rows, with 128 24.0 and 28.2, with 384 48.1 and 43.2. cols / 4 threads read a part; the groups of threads
// that share out the parts meet in shared memory, in a fixed order.
constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) q4_merge_kernel(const Q4AttnParams pp, int D,
                                                                 int cols, int row_tile, int C) {
    pdl_launch_dependents();
    pdl_wait();
    const RowsParams& p = pp.r;
    __shared__ float4 s_red[kMergeThreads];
    __shared__ float s_w[kQ4MaxShares], s_max[kMergeThreads / 32], s_sum[kMergeThreads / 32];
    const int rows_total = p.n_tok * p.G, tid = threadIdx.x;
    const int n_rt = (rows_total + row_tile - 1) / row_tile;
    const int slices = D / cols, slice = blockIdx.x % slices, R = blockIdx.x / slices;
    const int kvh = blockIdx.y, b = blockIdx.z, rt = R / row_tile;
    const int2 info = pp.info[(b * p.n_kv + kvh) * n_rt + rt];
    if (info.x < 0) return;  // one CTA took the whole unit and wrote its rows
    // parts: the second one of CTA info.x / 2 if info.x is odd, then the first ones up to CTA info.y
    const int c0 = info.x >> 1, nc = info.y - c0 + 1;
    if (info.y >= C || nc < 1) return;  // (a wait gave up, which is reported, and left the entry)
    auto part_row = [&](int c) {
        return ((size_t)(c ? 2 * (c0 + c) : info.x)) * row_tile + (R - rt * row_tile);
    };
    const float2* ml = reinterpret_cast<const float2*>(p.ml_part);
    float M = -INFINITY;
    for (int c = tid; c < nc; c += kMergeThreads) M = fmaxf(M, ml[part_row(c)].x);
    M = warp_max(M);
    if ((tid & 31) == 0) s_max[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) M = fmaxf(M, s_max[w]);
    float l = 0.f;
    for (int c = tid; c < nc; c += kMergeThreads) {
        const float2 x = ml[part_row(c)];
        const float w = exp2f(x.x - M);  // 0 for a part without keys of this row (kNoMax)
        s_w[c] = w;
        l = fmaf(w, x.y, l);
    }
    l = warp_sum(l);
    if ((tid & 31) == 0) s_sum[tid >> 5] = l;
    __syncthreads();
    const int tpg = cols / 4, n_grp = kMergeThreads / tpg, grp = tid / tpg, c4 = tid - grp * tpg;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = grp; c < nc; c += n_grp) {
        const float w = s_w[c];
        const float4 x =
            *reinterpret_cast<const float4*>(p.o_part + part_row(c) * D + slice * cols + c4 * 4);
        acc.x = fmaf(w, x.x, acc.x);
        acc.y = fmaf(w, x.y, acc.y);
        acc.z = fmaf(w, x.z, acc.z);
        acc.w = fmaf(w, x.w, acc.w);
    }
    s_red[tid] = acc;
    __syncthreads();
    if (grp == 0) {
        for (int h = 1; h < n_grp; ++h) {
            const float4 u = s_red[h * tpg + c4];
            acc.x += u.x;
            acc.y += u.y;
            acc.z += u.z;
            acc.w += u.w;
        }
        l = 0.f;
#pragma unroll
        for (int w = 0; w < kMergeThreads / 32; ++w) l += s_sum[w];
        const float il = 1.f / l;
        const int tok = R / p.G;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                  (((size_t)b * p.n_tok + tok) * p.n_q + kvh * p.G + R - tok * p.G) * D +
                                  slice * cols + c4 * 4) =
            make_uint2(pack_bf16(acc.x * il, acc.y * il), pack_bf16(acc.z * il, acc.w * il));
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

template <int D, int NQ, bool PAIR, bool CLUSTER>
cudaError_t launch(const Q4AttnParams& pp, int C, cudaStream_t st) {
    using L = Q4Layout<D>;
    Q4AttnParams p = pp;
    auto kernel = q4_attn_kernel<D, NQ, PAIR, CLUSTER>;
    static std::atomic<bool> configured[64];  // per device; the same value every time
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_relaxed);
    }
    // stages of the ring: as many as leave room for the other CTA of the SM, at least two
    constexpr int kFixed = 1024 + (kWarps / L::NG - 1) * 8 * NQ * D * 4;
    constexpr int kStatic = 2 * kT * (PAIR ? 16 : 8 * NQ) * 2 + kWarps * kT * 4 / (kWarps / L::NG) +
                            D / 16 * 32 * 2 * NQ * 4 + 2048;
    const int stage = (p.r.k_eq_v ? 1 : 2) * L::OP;
    int s = (112 * 1024 - kFixed - kStatic) / stage;
    s = s < 2 ? 2 : (s > kMaxStages ? kMaxStages : s);
    p.r.n_stages = s;
    const size_t smem = (size_t)kFixed + (size_t)s * stage;
    const uint64_t slots = p.r.page_size ? p.r.page_size : p.r.cap;
    const uint64_t rows = (uint64_t)(p.r.page_size ? p.r.n_pages : p.batch) * p.r.n_kv;
    CUtensorMap km, vm;
    if (!encode_codes(&km, p.r.k, L::ROWB, slots, rows) ||
        !encode_codes(&vm, p.r.v, L::ROWB, slots, rows))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, km, vm, p);
    if (e == cudaSuccess && p.balanced) {
        const int rows = p.r.n_tok * p.r.G;
        const int cols = (long long)rows * p.r.n_kv * p.batch >= 256 ? D : 64;
        e = launch_pdl(q4_merge_kernel, dim3((unsigned)(rows * (D / cols)), p.r.n_kv, p.batch),
                       dim3(kMergeThreads), 0, st, p, D, cols, 8 * NQ, C);
    }
    return e;
}

template <int D>
cudaError_t launch_d(const Q4AttnParams& p, int C, cudaStream_t st) {
    const int rows = p.r.n_tok * p.r.G;
    // (8 rows of 16 x 4096 keys: 18.7, 15.8, 13.0 us at head_dim 512, 256, 64; as 16: 22.1, 18.5, 15.2)
    if (rows > 8)
        return p.cluster > 1 ? launch<D, 2, false, true>(p, C, st)
                             : launch<D, 2, false, false>(p, C, st);
    if (rows > 4)
        return p.cluster > 1 ? launch<D, 1, false, true>(p, C, st)
                             : launch<D, 1, false, false>(p, C, st);
    return p.cluster > 1 ? launch<D, 1, true, true>(p, C, st)
                         : launch<D, 1, true, false>(p, C, st);
}

}  // namespace

cudaError_t launch_q4_attn(const RowsParams& r, const Q4Cache& c, int head_dim, int batch, int C,
                           int balanced, int cluster, void* info, cudaStream_t st) {
    const Q4AttnParams p{r, c.k_scales, c.v_codes ? c.v_scales : c.k_scales, batch, balanced,
                         cluster, static_cast<int2*>(info)};
    switch (head_dim) {
        case 64: return launch_d<64>(p, C, st);
        case 128: return launch_d<128>(p, C, st);
        case 256: return launch_d<256>(p, C, st);
        case 512: return launch_d<512>(p, C, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gemma
