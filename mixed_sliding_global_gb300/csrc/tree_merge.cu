// tree_merge.cu -- merge of the parts that the equal shares of tree_tc.cu and tree_pair.cu leave of a
// unit (one KV head of one sequence, a tile of rows, 256 columns at most):
//   M = max_w m_w, out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
// and zeros for row tiles without nodes. A lane has one row and 16 columns: parts lie with four columns of
// 128 rows after another, so reads are of 512 consecutive bytes, and writes are whole sectors. WAYS warps
// share out the parts (few units are cut into many), BATCH at a time, and meet in shared memory. Latency
// bound: a warp waits for memory twice (lengths, parts) where BATCH covers its parts.
#include "common.cuh"
#include "tree.h"
#include "tree_dev.cuh"

namespace gemma {

namespace {

// A unit in workers' parts: its key tiles are f0 .. f1 - 1 of all, `share` to a worker.
struct MergeUnit {
    int b, kvh, rt, half, f0, f1, share;
};

// 32 rows (from 32 * group on) and 16 columns of a unit; s_acc[8]: the ways' sums. Whole CTAs.
template <int D, int ROWS, int WAYS, int BATCH>
GEMMA_DEVINL void merge_rows(const MergeParams& mp, const MergeUnit& u, int group, int slice, int way,
                             float (*s_acc)[18][32]) {
    constexpr int COLS = D < 256 ? D : 256;  // of a piece: 128 rows x COLS
    constexpr int C = ROWS / 128;            // pieces of a part
    const RowsParams& p = mp.tp.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rr = group * 32 + lane, R = u.rt * ROWS + rr, c = rr >> 7, r = rr & 127;
    const int w0 = u.f0 / u.share, w1 = (u.f1 - 1) / u.share;
    float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    if (slice < D / 16) {
        for (int wb = w0 + way; wb <= w1; wb += BATCH * WAYS) {
            float2 ml[BATCH];
            float4 o[BATCH][4];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int w = wb + i * WAYS;
                // worker w's part is the first of its share but for one that began before the unit
                const size_t piece = (size_t)(2 * w + (w * u.share < u.f0)) * C + c;
                const float4* src = reinterpret_cast<const float4*>(mp.part_o) +
                                    (piece * (COLS / 4) + 4 * (slice % (COLS / 16))) * 128 + r;
                ml[i] = w <= w1 ? mp.part_ml[piece * 128 + r] : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[i][q] = w <= w1 ? __ldcs(src + q * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                top = fmaxf(top, ml[i].x);
                if (ml[i].x == -INFINITY) l += ml[i].y;  // (0; NaN where every score was)
            }
            if (top == -INFINITY) continue;
            const float a = fast_exp2(m - top);  // 0 while there was nothing
            m = top;
            l *= a;
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] *= a;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (ml[i].x == -INFINITY) continue;  // (no keys: O is nothing, or NaN where V is)
                const float e = fast_exp2(ml[i].x - top);
                l = fmaf(e, ml[i].y, l);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[4 * q] = fmaf(e, o[i][q].x, acc[4 * q]);
                    acc[4 * q + 1] = fmaf(e, o[i][q].y, acc[4 * q + 1]);
                    acc[4 * q + 2] = fmaf(e, o[i][q].z, acc[4 * q + 2]);
                    acc[4 * q + 3] = fmaf(e, o[i][q].w, acc[4 * q + 3]);
                }
            }
        }
    }
    if constexpr (WAYS > 1) {
        if (way) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s_acc[warp][e][lane] = acc[e];
            s_acc[warp][16][lane] = l;
            s_acc[warp][17][lane] = m;
        }
        __syncthreads();
        if (way) return;
        float top = m;
#pragma unroll
        for (int k = 1; k < WAYS; ++k) top = fmaxf(top, s_acc[warp + k][17][lane]);
        const float a = m == -INFINITY ? 0.f : fast_exp2(m - top);
        l *= a;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] *= a;
#pragma unroll
        for (int k = 1; k < WAYS; ++k) {
            const float mk = s_acc[warp + k][17][lane], ak = mk == -INFINITY ? 0.f : fast_exp2(mk - top);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = fmaf(ak, s_acc[warp + k][e][lane], acc[e]);
            l = fmaf(ak, s_acc[warp + k][16][lane], l);
        }
    }
    if (R >= p.n_tok * p.G || slice >= D / 16) return;
    const int tk = R / p.G;
    uint4* dst = reinterpret_cast<uint4*>(
        reinterpret_cast<__nv_bfloat16*>(p.out) +
        (((size_t)u.b * p.n_tok + tk) * p.n_q + u.kvh * p.G + (R - tk * p.G)) * (size_t)D + slice * 16);
    const float inv = 1.f / l;
    uint32_t out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)  // (no keys: zeros)
        out[e] = l == 0.f ? 0u : pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// Zeros for 32 rows (from 32 * group on) of row tile rt of a KV head: the whole CTA.
template <int D, int ROWS>
GEMMA_DEVINL void zero_rows(const RowsParams& p, int b, int kvh, int rt, int group) {
    const int R0 = rt * ROWS + 32 * group, n_rows = min(32, p.n_tok * p.G - R0);
    for (int i = threadIdx.x; i < n_rows * (D / 8); i += 256) {
        const int R = R0 + i / (D / 8), tk = R / p.G;
        uint4* dst = reinterpret_cast<uint4*>(
            reinterpret_cast<__nv_bfloat16*>(p.out) +
            (((size_t)b * p.n_tok + tk) * p.n_q + kvh * p.G + (R - tk * p.G)) * (size_t)D);
        dst[i % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace

// Few units: some CTAs for each.
template <int D, int ROWS, int WAYS, int BATCH>
__global__ void __launch_bounds__(256) tree_merge_kernel(const MergeParams mp) {
    pdl_launch_dependents();
    constexpr int COLS = D < 256 ? D : 256, HALVES = D / COLS;
    constexpr int SLICES = 8 / WAYS;                   // of 16 columns, per CTA
    constexpr int PER = (D / 16 + SLICES - 1) / SLICES, GROUPS = ROWS / 32;
    const RowsParams& p = mp.tp.p;
    const int warp = threadIdx.x >> 5, way = warp % WAYS;
    const int slice = (blockIdx.x % PER) * SLICES + warp / WAYS;
    const int x = blockIdx.x / PER, group = x % GROUPS, unit = x / GROUPS;
    __shared__ float s_acc[WAYS > 1 ? 8 : 1][18][32];
    const int per = mp.n_rt * p.n_kv, b = unit / per, kvh = unit % per / mp.n_rt,
              rt = unit % mp.n_rt;
    if (rt * ROWS + group * 32 >= p.n_tok * p.G) return;
    pdl_wait();  // the parts
    const int total = mp.before[mp.batch], whole = mp.before[mp.batch + 1], first = mp.before[b];
    const TrSeq sq = tr_seq(p, b);
    const int live_rt = sq.bad ? 0 : (sq.n * p.G + ROWS - 1) / ROWS;
    if (rt >= live_rt) {
        if (blockIdx.x % PER) return;
        if (sq.bad && rt == 0 && kvh == 0 && group == 0 && threadIdx.x == 0) report(p.err, sq.bad);
        zero_rows<D, ROWS>(p, b, kvh, rt, group);
        return;
    }
    if (whole) return;  // units were not cut
    const int nt = (sq.len - tr_start(p, sq) + mp.keys - 1) / mp.keys;
    const int share = (total + mp.workers - 1) / mp.workers, half = slice * 16 / COLS;
    const int f0 = first + ((kvh * live_rt + rt) * HALVES + half) * nt;
    const MergeUnit u{b, kvh, rt, half, f0, f0 + nt, share};
    if (f0 / share == (u.f1 - 1) / share) return;  // a whole unit: written by its worker
    merge_rows<D, ROWS, WAYS, BATCH>(mp, u, group, slice, way, s_acc);
}

// Many units: some CTAs for each place where a worker's share ends and another's begins, of
// which there are fewer, and the row tiles without nodes shared out among all CTAs.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) tree_merge_cuts_kernel(const MergeParams mp) {
    pdl_launch_dependents();
    constexpr int COLS = D < 256 ? D : 256, HALVES = D / COLS;
    constexpr int PER = (COLS / 16 + 7) / 8, GROUPS = ROWS / 32;
    const RowsParams& p = mp.tp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int x = blockIdx.x / PER, group = x % GROUPS, cut = x / GROUPS + 1;
    __shared__ float s_acc[8][18][32];
    pdl_wait();  // the parts
    const int total = mp.before[mp.batch], whole = mp.before[mp.batch + 1];
    for (long long i = blockIdx.x; i < (long long)mp.n_rt * mp.batch * p.n_kv * GROUPS; i += gridDim.x) {
        const int unit = (int)(i / GROUPS), g = (int)(i % GROUPS), per = mp.n_rt * p.n_kv;
        const int b = unit / per, kvh = unit % per / mp.n_rt, rt = unit % mp.n_rt;
        const TrSeq sq = tr_seq(p, b);
        if (rt < (sq.bad ? 0 : (sq.n * p.G + ROWS - 1) / ROWS)) continue;
        if (sq.bad && rt == 0 && kvh == 0 && g == 0 && threadIdx.x == 0) report(p.err, sq.bad);
        zero_rows<D, ROWS>(p, b, kvh, rt, g);
    }
    const int share = (total + mp.workers - 1) / mp.workers;
    const long long at = (long long)cut * share;
    if (whole || at >= total) return;
    // the sequence that holds the cut: the last one that begins at or before it and has tiles
    int b = 0;
    for (int lo = 0, n = mp.batch; n > 1;) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, lane * step < n && mp.before[i] <= at);
        const int k = 31 - __clz(in);
        lo += k * step;
        n = min(step, n - k * step);
        b = lo;
    }
    const TrSeq sq = tr_seq(p, b);
    const int live_rt = (sq.n * p.G + ROWS - 1) / ROWS,
              nt = (sq.len - tr_start(p, sq) + mp.keys - 1) / mp.keys;
    const int first = mp.before[b], idx = ((int)at - first) / nt, f0 = first + idx * nt;
    const MergeUnit u{b, idx / HALVES / live_rt, idx / HALVES % live_rt, idx % HALVES, f0, f0 + nt, share};
    // the unit's parts, and which of its cuts this is (-1: it begins there): the first `ways` of them share
    // out the columns, so that as many warps can share out the parts
    const int parts = (u.f1 - 1) / share - f0 / share + 1, nth = cut - f0 / share - 1;
    const int ways = parts < 5 ? 1 : parts < 10 ? 2 : parts < 24 ? 4 : 8;
    if (parts < 2 || nth < 0 || nth >= ways || u.rt * ROWS + group * 32 >= p.n_tok * p.G) return;
    const int slice0 = (blockIdx.x % PER) * 8 + nth * (8 / ways), slice = slice0 + warp / ways;
    if (slice0 >= COLS / 16) return;
    const int col = u.half * (COLS / 16) + slice;
    switch (ways) {
        case 1:
            if (slice < COLS / 16) merge_rows<D, ROWS, 1, 2>(mp, u, group, col, 0, s_acc);
            return;
        case 2: return merge_rows<D, ROWS, 2, 2>(mp, u, group, col, warp % 2, s_acc);
        case 4: return merge_rows<D, ROWS, 4, 2>(mp, u, group, col, warp % 4, s_acc);
    }
    merge_rows<D, ROWS, 8, 2>(mp, u, group, col, warp % 8, s_acc);
}

template <int D, int ROWS>
static cudaError_t launch_merge(const MergeParams& mp, cudaStream_t st) {
    const long long units = (long long)mp.n_rt * mp.batch * mp.tp.p.n_kv, groups = units * (ROWS / 32);
    // By the cuts where units are well above the workers: one by one they are more CTAs, and the parts that few
    // live sequences of a large batch leave want more warps than the host can know of. By units / by cuts: 224
    // units on 152 workers (head_dim 64, 17 tiles) 35.2 / 37.2 us; 128 on 76 (head_dim 256, 32 tiles) 120 /
    // 120, with one live sequence of the 64 31.5 / 20.1.
    if (2 * units * (D > 256 ? 2 : 1) > 3 * mp.workers) {
        constexpr int COLS = D < 256 ? D : 256;
        const int cuts = mp.workers > 1 ? mp.workers - 1 : 1;
        return launch_pdl(tree_merge_cuts_kernel<D, ROWS>,
                          dim3((unsigned)(cuts * (ROWS / 32) * ((COLS / 16 + 7) / 8))), dim3(256), 0, st, mp);
    }
    // Parts per unit, about, decide how many warps share them out and how many of them a warp has in flight;
    // while the CTAs are fewer than the SMs, twice the warps. In us of the whole step with 1 x 2, 2 x 2, 2 x
    // 4, 4 x 2, 4 x 4 and 8 x 4: 5 parts (14 units of 244 rows, head_dim 256) 24.7, 23.0, 24.7, 24.9, 26.8, -;
    // 9 (8 units of 256 rows, head_dim 512) 21.2, 18.6, 18.0, 19.2, 19.7, -; 9 (16 of 64, head_dim 128) 21.2,
    // 18.3, 17.4, 16.8, 16.4, -; 19 (4 of 256, head_dim 512) 28.6, 25.4, 24.0, 23.1, 22.4, -; 64 (one of 64,
    // head_dim 64) 20.6, 14.7, 13.3, 11.3, 10.7, 9.3.
    const long long parts = mp.workers / (units * (D > 256 ? 2 : 1));
    const long long warps = groups * (D / 16);
    int ways = parts < 5 ? 1 : parts < 10 ? 2 : parts < 24 ? 4 : 8;
    if (ways > 1 && ways < 8 && warps * ways < 8 * mp.tp.n_sm) ways *= 2;
    auto launch = [&](auto kernel, int slices) {
        return launch_pdl(kernel, dim3((unsigned)(groups * ((D / 16 + slices - 1) / slices))), dim3(256),
                          0, st, mp);
    };
    const bool four = parts >= 4 * ways;
    switch (ways) {
        case 1: return launch(tree_merge_kernel<D, ROWS, 1, 2>, 8);
        case 2: return launch(four ? tree_merge_kernel<D, ROWS, 2, 4> : tree_merge_kernel<D, ROWS, 2, 2>, 4);
        case 4: return launch(four ? tree_merge_kernel<D, ROWS, 4, 4> : tree_merge_kernel<D, ROWS, 4, 2>, 2);
    }
    return launch(tree_merge_kernel<D, ROWS, 8, 4>, 1);
}

cudaError_t launch_tree_merge(const MergeParams& mp, int head_dim, int rows, cudaStream_t st) {
    if (rows == 256) return head_dim == 256 ? launch_merge<256, 256>(mp, st) : launch_merge<512, 256>(mp, st);
    switch (head_dim) {
        case 64: return launch_merge<64, 128>(mp, st);
        case 128: return launch_merge<128, 128>(mp, st);
        case 256: return launch_merge<256, 128>(mp, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gemma
