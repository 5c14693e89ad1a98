// tree_dev.cuh -- what the attention kernels of a drafted tree share on the device: a sequence's
// lengths and key range, a node's ancestors, and its scores.
#pragma once

#include "common.cuh"
#include "tree.h"

namespace gemma {

constexpr int kTrWords = kTreeMaxNodes / 32;  // words of an ancestor set
constexpr float kTrLazyLog2 = 8.f;            // a row's reference moves past this growth only

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

// scale * dot, soft-capped where a cap is set, in log2 units. tanh through one exponential and one
// reciprocal: its absolute error (2^-22) times the cap is what the score is off by.
GEMMA_DEVINL float tr_score(const RowsParams& p, float dot) {
    if (p.softcap > 0.f) {
        const float e = fast_exp2(dot * p.cap_inner * 2.885390081777927f);  // exp(2 x)
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return fmaf(-2.f * p.cap_log2, r, p.cap_log2);
    }
    return dot * p.scale_log2;
}

}  // namespace gemma
