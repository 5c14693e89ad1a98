// kv_q4.cu -- writing and reading the rows of a 4-bit KV cache (format: q4.h).
//
// All three kernels move rows and are bound by the bytes (and, for a decode step's few rows, by
// the launch): a thread owns eight consecutive elements, i.e. one 32-bit code word, so a warp
// reads or writes 512 contiguous bytes of bf16 and 128 of codes; the eight threads of a group of
// 64 elements share its maximum through three shuffles.
#include "common.cuh"
#include "q4.h"

namespace gemma {

namespace {

constexpr int kThreads = 256;

struct Q4Rows {
    Q4Cache c;
    const void* src[2];   // append: new K, V rows [batch][n][n_kv][d]
    void* dst[2];         // read: rows out
    const int32_t* pos;   // first position per sequence (append, read)
    uint32_t* err;
    int batch, n, d_log2; // n rows per sequence
    // expand
    const int32_t* seq_lens;
    int32_t* lens_out;
    int n_tok, max_seq_len, window;
};

// Row index of position p in the [rows][slots] view of the cache; false for a bad page.
__device__ __forceinline__ bool q4_row(const Q4Cache& c, int b, int h, long long p, size_t& row) {
    if (c.pg.block_table) {
        const int blk = (int)(p / c.pg.page_size);
        const int page = __ldg(c.pg.block_table + (size_t)b * c.pg.max_pages + blk);
        row = ((size_t)page * c.n_kv + h) * (size_t)c.pg.page_size +
              (size_t)(p - (long long)blk * c.pg.page_size);
        return page >= 0 && page < c.pg.n_pages;
    }
    row = ((size_t)b * c.n_kv + h) * (size_t)c.cap + (size_t)(c.ring ? p % c.ring : p);
    return true;
}

// Smallest number of at most five significant bits, at least 2^-126, with 7 s >= amax > 0
// (finite), but no more than the largest whose 7 s is finite in bf16 (a maximum above that 7 s is
// less than 7.5 s, so its code is still 7). The reciprocal's rounding can miss by one step either
// way; 7 s is exact in fp32.
__device__ __forceinline__ float q4_scale(float amax) {
    constexpr uint32_t kStep = 0x00080000u;  // one unit of the fifth significant bit
    constexpr uint32_t kTop = 0x7e100000u;   // 1.125 * 2^125
    uint32_t u = __float_as_uint(amax * (1.f / 7.f)) & ~(kStep - 1);
    if (u < 0x00800000u) u = 0x00800000u;
    while (7.f * __uint_as_float(u) < amax && u < kTop) u += kStep;
    if (u > 0x00800000u && 7.f * __uint_as_float(u - kStep) >= amax) u -= kStep;
    return __uint_as_float(u);
}

// |x| / s rounded to the nearest integer, halves to even, s of five significant bits. The
// quotient of a bf16 |x| is a multiple of 2^-k / 31 for small k, so fp32 division never rounds a
// non-tie onto a tie; an fp32 |x| takes the division in 64 bits for the same property.
template <bool F32>
__device__ __forceinline__ uint32_t q4_code(float ax, float s) {
    if (F32) return (uint32_t)__double2int_rn((double)ax / (double)s);
    return (uint32_t)__float2int_rn(__fdiv_rn(ax, s));
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const Q4Rows p) {
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y, which = blockIdx.z;
    const int upr_log2 = p.d_log2 - 3;                    // units (8 elements) per row
    const uint32_t units = (uint32_t)p.n * p.c.n_kv << upr_log2;
    const int pos0 = __ldg(p.pos + b);
    if (pos0 < 0 || (!p.c.ring && (long long)pos0 + p.n > p.c.cap)) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && which == 0) report(p.err, GEMMA_DEVERR_WRITE_POS);
        return;
    }
    uint8_t* codes = which ? p.c.v_codes : p.c.k_codes;
    __nv_bfloat16* scales = which ? p.c.v_scales : p.c.k_scales;
    const uint32_t lane = threadIdx.x & 31;
    for (uint32_t base = blockIdx.x * kThreads + (threadIdx.x & ~31u); base < units;
         base += gridDim.x * kThreads) {
        const uint32_t unit = base + lane;
        const bool live = unit < units;  // a group's eight threads are all live or all not
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const size_t src = ((size_t)b * units + unit) * 8;
        if (live) {
            if (F32) {
                const float4* s4 = reinterpret_cast<const float4*>(
                    static_cast<const float*>(p.src[which]) + src);
                const float4 lo = __ldg(s4), hi = __ldg(s4 + 1);
                x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
                x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
            } else {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(p.src[which]) + src));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = __uint_as_float(w[i] << 16);
                    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        }
        // magnitudes as integers: their order is the numbers', with inf and NaN above all
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = max(mx, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (!live) continue;
        uint32_t word = 0;
        float s = 0.f;
        if (mx >= 0x7f800000u) {
            s = __uint_as_float(0x7fc00000u);
        } else if (mx > 0) {
            s = q4_scale(__uint_as_float(mx));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t sh = 16 * (e & 1) + 4 * (e >> 1);
                word |= q4_code<F32>(fabsf(x[e]), s) << sh;
                word |= (__float_as_uint(x[e]) >> 31) << ((sh + 15) & 31);
            }
        }
        const uint32_t row_in = unit >> upr_log2, u = unit & ((1u << upr_log2) - 1);
        const uint32_t t = row_in / (uint32_t)p.c.n_kv, h = row_in - t * p.c.n_kv;
        size_t row;
        if (!q4_row(p.c, b, (int)h, (long long)pos0 + t, row)) {
            if (u == 0 && h == 0) report(p.err, GEMMA_DEVERR_PAGE);
            continue;
        }
        *reinterpret_cast<uint32_t*>(codes + ((row << upr_log2) + u) * 4) = word;
        if ((u & 7) == 0)
            scales[(row << (upr_log2 - 3)) + (u >> 3)] = __float2bfloat16_rn(s);
    }
}

// The eight elements of a code word times the scale (exact).
__device__ __forceinline__ void q4_values(uint32_t word, float s, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t pr = __funnelshift_r(word, word, 4 * j) & 0x80078007u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t half = pr >> (16 * h);
            const float m = (float)(half & 7u) * s;
            x[2 * j + h] = half & 0x8000u ? -m : m;
        }
    }
}

template <bool F32>
__device__ __forceinline__ void q4_store(void* out, size_t elem, const float (&x)[8]) {
    if (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + elem);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + elem) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                       pack_bf16(x[6], x[7]));
    }
}

// EXPAND: positions from the first query's window start to the sequence's end, into
// [batch][n_kv][n][d]; else rows pos[b] + t into [batch][n][n_kv][d].
template <bool F32, bool EXPAND>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const Q4Rows p) {
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y, which = blockIdx.z;
    const int upr_log2 = p.d_log2 - 3;
    long long first;
    uint32_t rows = (uint32_t)p.n;
    bool bad = false;
    if (EXPAND) {
        const int len = __ldg(p.seq_lens + b);
        bad = len < p.n_tok || (!p.c.ring && len > p.c.cap) || len > p.max_seq_len;
        first = p.window ? max(0, len - p.n_tok - p.window + 1) : 0;
        if (blockIdx.x == 0 && threadIdx.x == 0 && which == 0)
            p.lens_out[b] = bad ? 0 : (int)(len - first);
        if (bad) return;  // reported by the attention launch, which sees length 0
        rows = (uint32_t)(len - first);
    } else {
        const int r0 = __ldg(p.pos + b);
        bad = r0 < 0 || (!p.c.ring && (long long)r0 + p.n > p.c.cap);
        first = r0;
        if (bad && blockIdx.x == 0 && threadIdx.x == 0 && which == 0)
            report(p.err, GEMMA_DEVERR_WRITE_POS);
    }
    const uint8_t* codes = which ? p.c.v_codes : p.c.k_codes;
    const __nv_bfloat16* scales = which ? p.c.v_scales : p.c.k_scales;
    const uint32_t units = rows * (uint32_t)p.c.n_kv << upr_log2;
    for (uint32_t unit = blockIdx.x * kThreads + threadIdx.x; unit < units;
         unit += gridDim.x * kThreads) {
        const uint32_t row_in = unit >> upr_log2, u = unit & ((1u << upr_log2) - 1);
        uint32_t t, h;
        if (EXPAND) {
            h = row_in / rows;
            t = row_in - h * rows;
        } else {
            t = row_in / (uint32_t)p.c.n_kv;
            h = row_in - t * p.c.n_kv;
        }
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        size_t row;
        if (!bad) {
            if (q4_row(p.c, b, (int)h, first + t, row)) {
                const uint32_t word =
                    __ldg(reinterpret_cast<const uint32_t*>(codes) + (row << upr_log2) + u);
                const float s = __bfloat162float(scales[(row << (upr_log2 - 3)) + (u >> 3)]);
                q4_values(word, s, x);
            } else if (u == 0 && h == 0) {
                report(p.err, GEMMA_DEVERR_PAGE);
            }
        }
        const size_t out_row = EXPAND ? ((size_t)b * p.c.n_kv + h) * (size_t)p.n + t
                                      : (size_t)b * p.n * p.c.n_kv + row_in;
        q4_store<F32>(p.dst[which], ((out_row << upr_log2) + u) * 8, x);
    }
}

int log2_of(int d) {
    int l = 0;
    while ((1 << l) < d) ++l;
    return l;
}

// grid of one launch over (units of a sequence, sequence, K / V): about eight CTAs per SM at most
dim3 q4_grid(long long rows, int n_kv, int head_dim, int batch, bool two, int n_sm) {
    const long long blocks = (rows * n_kv * (head_dim / 8) + kThreads - 1) / kThreads;
    long long limit = (long long)n_sm * 8 / ((long long)batch * (two ? 2 : 1));
    if (limit < 1) limit = 1;
    return dim3((unsigned)(blocks < limit ? (blocks < 1 ? 1 : blocks) : limit), (unsigned)batch,
                two ? 2 : 1);
}

}  // namespace

cudaError_t launch_q4_append(const Q4Cache& c, const void* k_new, const void* v_new,
                             const int32_t* write_pos, int batch, int n_new, int head_dim,
                             int fp32, uint32_t* err, int n_sm, cudaStream_t st) {
    Q4Rows p{};
    p.c = c;
    p.src[0] = k_new;
    p.src[1] = v_new;
    p.pos = write_pos;
    p.err = err;
    p.batch = batch;
    p.n = n_new;
    p.d_log2 = log2_of(head_dim);
    const dim3 grid = q4_grid(n_new, c.n_kv, head_dim, batch, c.v_codes != nullptr, n_sm);
    if (fp32) return launch_pdl(q4_append_kernel<true>, grid, dim3(kThreads), 0, st, p);
    return launch_pdl(q4_append_kernel<false>, grid, dim3(kThreads), 0, st, p);
}

cudaError_t launch_q4_read(const Q4Cache& c, void* k_out, void* v_out, const int32_t* read_pos,
                           int batch, int n_rows, int head_dim, int fp32, uint32_t* err, int n_sm,
                           cudaStream_t st) {
    Q4Rows p{};
    p.c = c;
    p.dst[0] = k_out;
    p.dst[1] = v_out;
    p.pos = read_pos;
    p.err = err;
    p.batch = batch;
    p.n = n_rows;
    p.d_log2 = log2_of(head_dim);
    const dim3 grid = q4_grid(n_rows, c.n_kv, head_dim, batch, c.v_codes != nullptr, n_sm);
    if (fp32) return launch_pdl(q4_read_kernel<true, false>, grid, dim3(kThreads), 0, st, p);
    return launch_pdl(q4_read_kernel<false, false>, grid, dim3(kThreads), 0, st, p);
}

cudaError_t launch_q4_expand(const Q4Cache& c, void* k_out, void* v_out, int32_t* lens_out,
                             const int32_t* seq_lens, int batch, int n_tok, int max_seq_len,
                             int window, int slots, int head_dim, uint32_t* err, int n_sm,
                             cudaStream_t st) {
    Q4Rows p{};
    p.c = c;
    p.dst[0] = k_out;
    p.dst[1] = v_out;
    p.err = err;
    p.batch = batch;
    p.n = slots;
    p.d_log2 = log2_of(head_dim);
    p.seq_lens = seq_lens;
    p.lens_out = lens_out;
    p.n_tok = n_tok;
    p.max_seq_len = max_seq_len;
    p.window = window;
    const dim3 grid = q4_grid(slots, c.n_kv, head_dim, batch, c.v_codes != nullptr, n_sm);
    return launch_pdl(q4_read_kernel<false, true>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace gemma
