// tree_dev.cuh -- what the attention kernels of a drafted tree share on the device: a sequence's
// lengths and key range, a node's ancestors, and its scores.
#pragma once

#include <cuda.h>

#include <climits>

#include "common.cuh"
#include "tc.cuh"
#include "tree.h"

namespace gemma {

constexpr int kTrWords = kTreeMaxNodes / 32;  // words of an ancestor set
constexpr float kTrLazyLog2 = 8.f;            // a row's reference moves past this growth only
constexpr float kTrPlainCap = 64.f;           // caps with one form of tanh per thread (tree_cap)

// Barrier of n threads that tells each whether v is true for any.
GEMMA_DEVINL bool named_bar_or(int id, int n, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

// A sequence's lengths. bad: an error bit, the sequence has no rows.
struct TrSeq {
    int len, n, base;
    uint32_t bad;
};
GEMMA_DEVINL TrSeq tr_seq(const RowsParams& p, int b) {
    TrSeq s;
    s.len = __ldg(p.seq_lens + b);
    s.n = p.n_real ? __ldg(p.n_real + b) : p.n_tok;
    s.bad = 0;
    if (s.n < 0 || s.n > p.n_tok) s.bad = GEMMA_DEVERR_N_REAL;
    else if (s.len < s.n || (!p.ring && s.len > p.cap) || s.len > p.max_seq_len)
        s.bad = GEMMA_DEVERR_SEQ_LEN;
    s.base = s.len - s.n;
    return s;
}
// First key that any node may attend, and where the chunks start (rings and pages: whole tiles).
GEMMA_DEVINL int tr_first(const RowsParams& p, const TrSeq& s) {
    return p.is_sliding ? max(0, s.base - p.window + 1) : 0;
}
GEMMA_DEVINL int tr_start(const RowsParams& p, const TrSeq& s) {
    const int first = tr_first(p, s);
    return p.ring || p.page_size ? first & ~(kTreeKeyTile - 1) : first;
}
// Chunks of a sequence that hold keys.
GEMMA_DEVINL int tr_chunks(const RowsParams& p, const TrSeq& s) {
    return min(p.n_split, (s.len - tr_start(p, s) + p.chunk - 1) / p.chunk);
}

// Walks from node i to the root: the set of the nodes it attends, and its depth. par: validated.
GEMMA_DEVINL int tr_walk(const int* par, int i, int window, uint32_t (&set)[kTrWords]) {
#pragma unroll
    for (int w = 0; w < kTrWords; ++w) set[w] = 0;
    int depth = 0;
    for (int m = i; m >= 0; m = par[m], ++depth)
        if (depth < window) {
#pragma unroll
            for (int w = 0; w < kTrWords; ++w)
                if (w == m >> 5) set[w] |= 1u << (m & 31);
        }
    return depth - 1;
}

// Which of 64 consecutive keys a row attends: bit e is key e of a tile whose key 0 is node m0 (negative:
// a prefix key, the prefix ends at key -m0); prefix keys count from column lo on.
GEMMA_DEVINL unsigned long long tr_window(const uint32_t (&anc)[kTrWords], int m0, int lo) {
    unsigned long long see = 0;
    if (m0 >= 0) {
#pragma unroll
        for (int k = 0; k < kTrWords; ++k) {
            const int sh = m0 - 32 * k;  // right by sh, or left
            const unsigned long long x = anc[k];
            if (sh > -64 && sh < 32) see |= sh >= 0 ? x >> sh : x << -sh;
        }
        return see;
    }
    if (m0 > -64) see = ((unsigned long long)anc[1] << 32 | anc[0]) << -m0;
    const int end = min(64, -m0);
    if (lo < end) {
        const unsigned long long upto = end == 64 ? ~0ull : (1ull << end) - 1;
        see |= lo > 0 ? upto & ~((1ull << lo) - 1) : upto;
    }
    return see;
}

// tanh(x) / x by its Taylor series to x^11, of u = x^2: the first term left out is 0.0036 x^12, below
// 2^-20 for |x| <= 1/2.
constexpr float kTanh3 = -1.f / 3.f, kTanh5 = 2.f / 15.f, kTanh7 = -17.f / 315.f, kTanh9 = 62.f / 2835.f,
                kTanh11 = -1382.f / 155925.f;
GEMMA_DEVINL float tr_tanh_over_x(float u) {
    return fmaf(fmaf(fmaf(fmaf(fmaf(kTanh11, u, kTanh9), u, kTanh7), u, kTanh5), u, kTanh3), u, 1.f);
}
// scale * dot, soft-capped where a cap is set, in log2 units: cap * tanh(x), x = scale * dot / cap. Above
// |x| = 1/2 tanh goes through one exponential and one reciprocal; below, its absolute error there (2^-22,
// times the cap) would be large against the score, and the series takes its place.
GEMMA_DEVINL float tr_score(const RowsParams& p, float dot) {
    const float s = dot * p.scale_log2;
    if (p.softcap > 0.f) {
        const float x = dot * p.cap_inner, e = fast_exp2(x * 2.885390081777927f);  // exp(2 x)
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return fabsf(x) <= 0.5f ? s * tr_tanh_over_x(x * x) : fmaf(-2.f * p.cap_log2, r, p.cap_log2);
    }
    return s;
}

// A unit (one KV head of one sequence, a tile of ROWS rows, one of HALVES parts of head_dim), or a part
// of its keys.
struct TreeUnit {
    int b, kvh, rt, half;
    TrSeq sq;
    int first;             // first key that a node may attend
    int k_begin, n_tiles;  // the part's
    int slot;              // workspace slot, -1: the whole unit
};

// A sequence's tiles of KEYS keys per unit, and its row tiles that have rows.
template <int KEYS, int ROWS>
GEMMA_DEVINL int tree_tiles(const RowsParams& p, const TrSeq& s, int& live_rt) {
    live_rt = s.bad ? 0 : (s.n * p.G + ROWS - 1) / ROWS;
    return live_rt ? (s.len - tr_start(p, s) + KEYS - 1) / KEYS : 0;
}

// Place in a ring of slots: the slot, and how often the ring has been gone round.
struct TreeRing {
    int slot = 0, use = 0;
    GEMMA_DEVINL void step(int n) {
        if (++slot == n) {
            slot = 0;
            ++use;
        }
    }
};

// A worker's parts: the key tiles of all units, in the order of (sequence, KV head, row tile, half,
// keys), in equal shares. Whole warps run it alike, each by itself: lengths are known on the device
// alone, and this way no warp waits for another. Units are not cut where they are at most as many as
// the workers and the longest alone (tile_ns a tile) takes no longer than an equal share (share_ns a
// tile, when every SM works) and the merge of its parts (merge_ns). WHOLE: they never are, and of more
// units than workers a worker takes those that begin in its share.
template <int KEYS, int ROWS, int HALVES, bool WHOLE>
struct TreeShare {
    int pos, end, begin, b, seq0, worker;  // seq0: tiles (whole units) of the sequences before b
    bool whole;  // a worker has one unit
    GEMMA_DEVINL void init(const MergeParams& mp, int worker_, bool write_before, int tile_ns,
                           int share_ns, int merge_ns) {
        // lane l has the sequences l * per .. + per - 1: one round of loads for many of them
        const RowsParams& p = mp.tp.p;
        const int lane = threadIdx.x & 31, per = (mp.batch + 31) / 32;
        const int b_lo = min(mp.batch, lane * per), b_hi = min(mp.batch, b_lo + per);
        int n = 0, u = 0, longest = 0;
#pragma unroll 4
        for (int x = b_lo; x < b_hi; ++x) {
            int live_rt;
            const int nt = tree_tiles<KEYS, ROWS>(p, tr_seq(p, x), live_rt);
            n += nt * live_rt * p.n_kv * HALVES;
            u += live_rt * p.n_kv * HALVES;
            longest = max(longest, nt);
        }
        int n_incl = n, u_incl = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, n_incl, o),
                      z = __shfl_up_sync(0xffffffffu, u_incl, o);
            if (lane >= o) {
                n_incl += y;
                u_incl += z;
            }
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        const int total = __shfl_sync(0xffffffffu, n_incl, 31),
                  units = __shfl_sync(0xffffffffu, u_incl, 31);
        const int share = (total + mp.workers - 1) / mp.workers;
        whole = units <= mp.workers &&
                (WHOLE || (long long)longest * tile_ns <= (long long)share * share_ns + merge_ns);
        if (write_before) {
            int sum = n_incl - n;
            for (int x = b_lo; x < b_hi; ++x) {
                mp.before[x] = sum;
                int live_rt;
                sum += tree_tiles<KEYS, ROWS>(p, tr_seq(p, x), live_rt) * live_rt * p.n_kv * HALVES;
            }
            if (lane == 0) {
                mp.before[mp.batch] = total;
                mp.before[mp.batch + 1] = whole;
            }
        }
        worker = worker_;
        const int all = whole ? units : total, step = whole ? 1 : share;
        begin = pos = min(all, worker * step);
        end = min(all, pos + step);
        // next() goes on from the first sequence of the lane that holds pos
        const int incl = whole ? u_incl : n_incl;
        const unsigned in = __ballot_sync(0xffffffffu, incl > pos);
        const int l = in ? __ffs(in) - 1 : 0;
        b = l * per;
        seq0 = __shfl_sync(0xffffffffu, whole ? u_incl - u : n_incl - n, l);
    }
    GEMMA_DEVINL bool next(const MergeParams& mp, TreeUnit& U) {
        if (pos >= end) return false;
        const RowsParams& p = mp.tp.p;
        for (;; ++b) {  // (sequences without tiles are passed over)
            U.sq = tr_seq(p, b);
            int live_rt;
            const int nt = tree_tiles<KEYS, ROWS>(p, U.sq, live_rt), unit = whole ? 1 : nt,
                      all = unit * live_rt * p.n_kv * HALVES;
            if (WHOLE && !whole && nt > 0 && pos < seq0 + all) {  // on to where a unit begins
                pos = seq0 + (pos - seq0 + nt - 1) / nt * nt;
                if (pos >= end) return false;
            }
            if (pos < seq0 + all) {
                const int rel = pos - seq0, idx = whole ? rel : rel / nt, t0 = rel - idx * unit;
                const int t1 = whole || WHOLE ? nt : min(nt, t0 + end - pos);
                U.b = b;
                U.half = idx % HALVES;
                // Whole units: the KV heads of a row tile one after another, whose rows have the same ancestors
                // (552 units of 3 tiles, head_dim 64, 56 -> 43 us); else the row tiles of a KV head, which read
                // the same keys.
                if (WHOLE) {
                    U.rt = idx / HALVES / p.n_kv;
                    U.kvh = idx / HALVES - U.rt * p.n_kv;
                } else {
                    U.kvh = idx / HALVES / live_rt;
                    U.rt = idx / HALVES - U.kvh * live_rt;
                }
                U.first = tr_first(p, U.sq);
                U.k_begin = tr_start(p, U.sq) + t0 * KEYS;
                U.n_tiles = t1 - t0;
                U.slot = t0 == 0 && t1 == nt ? -1 : 2 * worker + (pos != begin);
                pos += whole ? 1 : t1 - t0;
                return true;
            }
            seq0 += all;
        }
    }
};

// One unit, or the part of its keys that CTA k of n takes: what a worker does where units are dealt out by
// the host.
template <int KEYS, int ROWS, int HALVES>
struct TreeAlone {
    TreeUnit U;
    bool more;
    GEMMA_DEVINL void init(const MergeParams& mp, int unit, int k, int n) {
        const RowsParams& p = mp.tp.p;
        U.half = unit % HALVES;
        unit /= HALVES;
        const int per = mp.n_rt * p.n_kv;
        U.b = unit / per;
        U.kvh = unit % per / mp.n_rt;
        U.rt = unit % mp.n_rt;
        U.slot = -1;
        U.sq = tr_seq(p, U.b);
        int live_rt;
        int nt = tree_tiles<KEYS, ROWS>(p, U.sq, live_rt);
        if (U.rt >= live_rt) nt = 0;
        const int t0 = nt * k / n;
        U.first = tr_first(p, U.sq);
        U.k_begin = tr_start(p, U.sq) + t0 * KEYS;
        U.n_tiles = nt * (k + 1) / n - t0;
        more = U.n_tiles > 0;
    }
    GEMMA_DEVINL bool next(const MergeParams&, TreeUnit& X) {
        X = U;
        const bool now = more;
        more = false;
        return now;
    }
};

// Row tiles without nodes: zeros, an eighth of a tile at a time, and bad lengths are reported. One warp of
// each of `workers` CTAs, in turn.
template <int D, int ROWS>
GEMMA_DEVINL void tree_dead_rows(const MergeParams& mp, int worker, int workers) {
    const RowsParams& p = mp.tp.p;
    const int lane = threadIdx.x & 31;
    for (long long i = worker; i < 8ll * mp.n_rt * mp.batch; i += workers) {
        const int b = (int)(i / (8 * mp.n_rt)), rt = (int)(i / 8 % mp.n_rt), eighth = (int)(i % 8);
        const TrSeq sq = tr_seq(p, b);
        if (rt < (sq.bad ? 0 : (sq.n * p.G + ROWS - 1) / ROWS)) continue;
        if (sq.bad && rt == 0 && eighth == 0 && lane == 0) report(p.err, sq.bad);
        // (tokens with all their heads: 8 G divides ROWS)
        const int toks = ROWS / p.G / 8, tok0 = rt * (ROWS / p.G) + eighth * toks,
                  n_tok = min(toks, p.n_tok - tok0);
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) +
                                              ((size_t)b * p.n_tok + tok0) * p.n_q * (size_t)D);
        const long long n = (long long)n_tok * p.n_q * (D / 8);
        for (long long k = lane; k < n; k += 32) dst[k] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// What a row attends: its ancestors, and the first prefix key. Whole warps; every warp of a sequence
// finds a bad tree by itself.
struct TreeRow {
    uint32_t anc[kTrWords];
    int lo;  // INT_MAX: the row attends nothing
    GEMMA_DEVINL void find(const TreeParams& tp, const TreeUnit& U, int R, bool reports) {
        const RowsParams& p = tp.p;
        const int lane = threadIdx.x & 31;
        const int32_t* par = tp.parents + (size_t)U.b * p.n_tok;
        bool bad = false;
        unsigned next[kTrWords];  // the nodes that follow their parents
#pragma unroll
        for (int k = 0; k < kTrWords; ++k) {
            const int i = lane + 32 * k, m = i < U.sq.n ? __ldg(par + i) : -1;
            anc[k] = 0;
            bad |= m < -1 || m >= i;
            next[k] = __ballot_sync(0xffffffffu, i > 0 && m == i - 1);
        }
        bad = __any_sync(0xffffffffu, bad);
        if (bad && reports) report(p.err, GEMMA_DEVERR_TREE);
        lo = INT_MAX;
        if (R >= U.sq.n * p.G || bad) return;
        // Up to the root, a run of nodes s .. m that follow their parents at a time: one by one a chain of 91 is
        // 1.9 us of dependent loads (552 units of 3 tiles, head_dim 64, chains 61 / 41 us; random trees 43 / 44).
        const int window = p.is_sliding ? p.window : INT_MAX;
        const unsigned long long n0 = next[0] | (unsigned long long)next[1] << 32,
                                 n1 = next[2] | (unsigned long long)next[3] << 32;
        auto below = [](int x) { return x <= 0 ? 0ull : x >= 64 ? ~0ull : (1ull << x) - 1; };
        unsigned long long a0 = 0, a1 = 0;
        int depth = 0;
        for (int m = R / p.G; m >= 0;) {
            const unsigned long long z1 = ~n1 & below(m - 63), z0 = ~n0 & below(m + 1);
            const int s = z1 ? 127 - __clzll((long long)z1) : 63 - __clzll((long long)z0);
            const int from = max(s, m + 1 - max(0, window - depth));
            a0 |= below(m + 1) & ~below(from);
            a1 |= below(m - 63) & ~below(from - 64);
            depth += m - s + 1;
            m = __ldg(par + s);
        }
        anc[0] = (uint32_t)a0;
        anc[1] = (uint32_t)(a0 >> 32);
        anc[2] = (uint32_t)a1;
        anc[3] = (uint32_t)(a1 >> 32);
        lo = p.is_sliding ? max(0, U.sq.base + depth - p.window) : 0;
    }
};

// 32 bytes (a whole sector) from one thread; 32-byte aligned
GEMMA_DEVINL void st_global_v8(void* dst, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 32 consecutive columns of a row of the output, O / l (zeros without keys, whatever the other rows' V
// holds); wide: `out` is 32-byte aligned
GEMMA_DEVINL void tree_store32(__nv_bfloat16* out, const uint32_t (&v)[32], float l, bool wide) {
    const float inv = 1.f / l;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = l == 0.f ? 0u
                            : pack_bf16(__uint_as_float(v[16 * q + 2 * e]) * inv,
                                        __uint_as_float(v[16 * q + 2 * e + 1]) * inv);
        if (wide) {
            st_global_v8(out + q * 16, w);
        } else {
            uint4* dst = reinterpret_cast<uint4*>(out + q * 16);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}
// N scores of a row soft-capped, in log2 units (tr_score); a NaN may spread to the score beside it. Three
// forms of tanh, by the thread's scores, so that a score's error is small against the row's largest score or
// against itself:
//  - up to |x| = 1/8 (in the whole warp) the series' first three terms, the next being 0.054 x^6 < 2^-22;
//  - up to 1/2 the series;
//  - above, 1 - 2 / (1 + e^2x), two scores to a reciprocal: off by at most 2^-20 of the cap. With the
//    softmax's own exponential 5 special-function instructions for two scores, which bound such a tile.
//    Up to a cap of 64 that is 2^-14 of a weight, 1/64 of what P's rounding may move it by; above, it is
//    small against the row's largest score where one of the thread's is above 0.46 of the cap before the
//    tanh, and where none is (keys far below the others) scores up to 1/2 take the series one by one. 76
//    units of 4096 keys, head_dim 256, so / with that choice for every cap, in us: a cap of 8 times the
//    scores 89 / 125, of twice 86 / 130.
template <int N>
GEMMA_DEVINL void tree_cap(float (&s)[N], const RowsParams& p) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < N; e += 2) top = fmax3f(top, fabsf(s[e]), fabsf(s[e + 1]));
    top *= p.cap_inner;
    const float k = p.scale_log2;
    const unsigned long long in = f32x2(p.cap_inner, p.cap_inner), c5 = f32x2(k * kTanh5, k * kTanh5),
                             c3 = f32x2(k * kTanh3, k * kTanh3), c1 = f32x2(k, k);
    if (__all_sync(0xffffffffu, top <= 0.125f)) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const unsigned long long v = f32x2(s[e], s[e + 1]), x = mul_f32x2(v, in), u = mul_f32x2(x, x);
            const float2 y = f32x2_split(mul_f32x2(v, fma_f32x2(fma_f32x2(c5, u, c3), u, c1)));
            s[e] = y.x;
            s[e + 1] = y.y;
        }
    } else if (top <= 0.5f) {
        const unsigned long long c11 = f32x2(k * kTanh11, k * kTanh11), c9 = f32x2(k * kTanh9, k * kTanh9),
                                 c7 = f32x2(k * kTanh7, k * kTanh7);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const unsigned long long v = f32x2(s[e], s[e + 1]), x = mul_f32x2(v, in), u = mul_f32x2(x, x);
            unsigned long long t = fma_f32x2(c11, u, c9);
            t = fma_f32x2(t, u, c7);
            t = fma_f32x2(t, u, c5);
            t = fma_f32x2(t, u, c3);
            const float2 y = f32x2_split(mul_f32x2(v, fma_f32x2(t, u, c1)));
            s[e] = y.x;
            s[e + 1] = y.y;
        }
    } else {
        const float in2 = 2.885390081777927f * p.cap_inner;  // exp(2 x) = 2^(in2 s)
        auto two = [&](float& s0, float& s1) {
            // (2^58 at most, so that the product of two stays in range; a NaN stays one)
            float x = s0 * in2, y = s1 * in2;
            x = x > 58.f ? 58.f : x;
            y = y > 58.f ? 58.f : y;
            const float a = 1.f + fast_exp2(x), b = 1.f + fast_exp2(y);
            float q;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(a * b));
            q *= -2.f * p.cap_log2;
            s0 = fmaf(q, b, p.cap_log2);
            s1 = fmaf(q, a, p.cap_log2);
        };
        bool apart = false;
        if (p.softcap > kTrPlainCap) {
            float hi = s[0];
#pragma unroll
            for (int e = 0; e < N; e += 2) hi = fmax3f(hi, s[e], s[e + 1]);
            apart = !(hi * p.cap_inner >= 0.46f);
        }
        if (!apart) {
#pragma unroll
            for (int e = 0; e < N; e += 2) two(s[e], s[e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const float s0 = s[e], s1 = s[e + 1], x = s0 * p.cap_inner, y = s1 * p.cap_inner;
                two(s[e], s[e + 1]);
                if (fabsf(x) <= 0.5f) s[e] = s0 * k * tr_tanh_over_x(x * x);
                if (fabsf(y) <= 0.5f) s[e + 1] = s1 * k * tr_tanh_over_x(y * y);
            }
        }
    }
    __syncwarp();
}
// Maximum of N scores (32 or 64).
template <int N>
GEMMA_DEVINL float tree_max(const float (&s)[N]) {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmax3f(s[i], s[8 + i], s[16 + i]);
#pragma unroll
    for (int e = 24; e + 8 < N; e += 16)
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = fmax3f(m[i], s[e + i], s[e + 8 + i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], s[N - 8 + i]);
    return fmax3f(fmax3f(m[0], m[1], m[2]), fmax3f(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}
// P = 2^(s * scale + neg) of N scores as packed bf16; returns their sum, as rounded.
template <int N>
GEMMA_DEVINL float tree_exp(const float (&s)[N], float scale, float neg, uint32_t (&pw)[N / 2]) {
    const unsigned long long scale2 = f32x2(scale, scale), neg2 = f32x2(neg, neg);
    unsigned long long sum[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float2 x = f32x2_split(fma_f32x2(f32x2(s[2 * k], s[2 * k + 1]), scale2, neg2));
        pw[k] = pack_bf16(fast_exp2(x.x), fast_exp2(x.y));
        sum[k & 1] = add_f32x2(sum[k & 1], f32x2(__uint_as_float(pw[k] << 16),
                                                 __uint_as_float(pw[k] & 0xffff0000u)));
    }
    const float2 a = f32x2_split(sum[0]), b = f32x2_split(sum[1]);
    return (a.x + a.y) + (b.x + b.y);
}
// Scores of keys that a row does not attend become x: N of them (32 or 64), key 0 is kt0.
template <int N>
GEMMA_DEVINL void tree_mask(float (&s)[N], const TreeRow& row, int kt0, int base, float x) {
    if (kt0 >= row.lo && kt0 + N <= base) return;
    const unsigned long long see = tr_window(row.anc, kt0 - base, row.lo - kt0);
    const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        if (!((s0 >> e) & 1u)) s[e] = x;
        if constexpr (N == 64)
            if (!((s1 >> e) & 1u)) s[32 + e] = x;
    }
}
// Packed P of 32 or 64 keys into tensor memory.
GEMMA_DEVINL void tmem_store(uint32_t addr, const uint32_t (&v)[32]) { tmem_st32(addr, v); }
GEMMA_DEVINL void tmem_store(uint32_t addr, const uint32_t (&v)[16]) { tmem_st16(addr, v); }
GEMMA_DEVINL void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

}  // namespace gemma
