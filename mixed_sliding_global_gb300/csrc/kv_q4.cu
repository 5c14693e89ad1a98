// kv_q4.cu -- writing and reading the rows of a 4-bit KV cache (format: q4.h).
//
// All three kernels move rows and are bound by the bytes (and, for a decode step's few rows, by
// the launch): a thread owns eight consecutive elements, i.e. one 32-bit code word, so a warp
// reads or writes 512 contiguous bytes of bf16 and 128 of codes; the eight threads of a group of
// 64 elements share its maximum through three shuffles. A thread keeps four units in flight: 4 x 512
// tokens of 8 x 256 elements, K and V, append and read back, take 15.2 us together (42.5 MB, 2.8
// TB/s; 20.7 with one unit in flight and a division per element). The integer pipe is then 55% busy in the append and 44% in
// the read-back, with 70% and 58% of the cycles issuing. One token of 64 sequences: 4.3 us for
// both, two launches of 1.3 MB.
#include "common.cuh"
#include "q4.h"

namespace gemma {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // units of a thread in flight: the rows come from DRAM

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
    int kv_log2;          // log2 of n_kv, or -1
    // row of a [n][n_kv] array to its token and KV head
    __device__ __forceinline__ void split(uint32_t row, uint32_t& t, uint32_t& h) const {
        t = kv_log2 >= 0 ? row >> kv_log2 : row / (uint32_t)c.n_kv;
        h = row - t * c.n_kv;
    }
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
// quotient of a bf16 |x| is a multiple of 2^-k / 31 for small k, so anything near enough tells
// non-ties apart, and a tie (an exact binary fraction) is what one correction of |x| * (1 / s) gives
// exactly: the residual is exact and the corrected quotient is off by less than half a unit. An
// IEEE division per element cost three times the rest of the kernel. fp32 |x| takes the division
// in 64 bits.
template <bool F32>
__device__ __forceinline__ uint32_t q4_code(float ax, float s, float inv) {
    if (F32) return (uint32_t)__double2int_rn((double)ax / (double)s);
    const float y = __fmul_rn(ax, inv);
    const float q = __fmaf_rn(__fmaf_rn(-y, s, ax), inv, y);
    return __float_as_uint(__fadd_rn(q, 12582912.f));  // 1.5 * 2^23: the integer in the low 16 bits
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
    // kAhead units per thread in flight (a whole group's threads are live or none)
    for (uint32_t base = blockIdx.x * (kThreads * kAhead) + threadIdx.x; base - (threadIdx.x & 31u) < units;
         base += gridDim.x * (kThreads * kAhead)) {
        uint4 raw[kAhead][F32 ? 2 : 1];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const uint32_t unit = base + a * kThreads;
            const size_t src = ((size_t)b * units + unit) * (F32 ? 2 : 1);
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i) {
                raw[a][i] = make_uint4(0u, 0u, 0u, 0u);
                if (unit < units)
                    raw[a][i] = reinterpret_cast<const uint4*>(p.src[which])[src + i];
            }
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const uint32_t unit = base + a * kThreads;
            uint32_t w[F32 ? 8 : 4];
#pragma unroll
            for (int i = 0; i < (F32 ? 2 : 1); ++i) {
                w[4 * i] = raw[a][i].x;
                w[4 * i + 1] = raw[a][i].y;
                w[4 * i + 2] = raw[a][i].z;
                w[4 * i + 3] = raw[a][i].w;
            }
            // magnitudes as integers: their order is the numbers', with inf and NaN above all
            uint32_t mx = 0;
#pragma unroll
            for (int e = 0; e < (F32 ? 8 : 4); ++e)
                mx = F32 ? max(mx, w[e] & 0x7fffffffu)
                         : max(mx, max(w[e] << 16 & 0x7fff0000u, w[e] & 0x7fff0000u));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (unit >= units) continue;
            uint32_t word = 0;
            float s = 0.f;
            if (mx >= 0x7f800000u) {
                s = __uint_as_float(0x7fc00000u);
            } else if (mx > 0) {
                s = q4_scale(__uint_as_float(mx));
                const float inv = __frcp_rn(s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // slot j: elements 2 j and 2 j + 1
                    const float x0 = __uint_as_float(F32 ? w[(2 * j) & 7] : w[j] << 16);
                    const float x1 = __uint_as_float(F32 ? w[(2 * j + 1) & 7] : w[j] & 0xffff0000u);
                    // magnitudes in the halves' low bits, signs on their top ones; the signs then
                    // rotate across the word's end, the magnitudes do not reach it
                    const uint32_t m = __byte_perm(q4_code<F32>(fabsf(x0), s, inv),
                                                   q4_code<F32>(fabsf(x1), s, inv), 0x5410);
                    const uint32_t sg = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632) &
                                        0x80008000u;
                    word |= m << (4 * j) | __funnelshift_l(sg, sg, 4 * j);
                }
            }
            const uint32_t row_in = unit >> upr_log2, u = unit & ((1u << upr_log2) - 1);
            uint32_t t, h;
            p.split(row_in, t, h);
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
}

// Slot j of a code word times the scale, as a bf16 pair: 128 + m is m in the low bits of bf16's 128,
// m and m * scale are exact, and the sign is put in front.
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, uint32_t scale2, int j) {
    const uint32_t r = __funnelshift_r(word, word, 4 * j);
    uint32_t v = (r & 0x00070007u) | 0x43004300u;
    asm("{\n\t.reg .b32 t;\n\tsub.rn.bf16x2 t, %0, %1;\n\tmul.rn.bf16x2 %0, t, %2;\n\t}"
        : "+r"(v)
        : "r"(0x43004300u), "r"(scale2));
    return v ^ (r & 0x80008000u);
}

template <bool F32>
__device__ __forceinline__ void q4_store(void* out, size_t elem, uint32_t word, uint32_t scale) {
    const uint32_t scale2 = scale * 0x10001u;
    const uint32_t v0 = q4_pair(word, scale2, 0), v1 = q4_pair(word, scale2, 1);
    const uint32_t v2 = q4_pair(word, scale2, 2), v3 = q4_pair(word, scale2, 3);
    if (F32) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<float*>(out) + elem);
        o[0] = make_uint4(v0 << 16, v0 & 0xffff0000u, v1 << 16, v1 & 0xffff0000u);
        o[1] = make_uint4(v2 << 16, v2 & 0xffff0000u, v3 << 16, v3 & 0xffff0000u);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + elem) =
            make_uint4(v0, v1, v2, v3);
    }
}

// EXPAND: positions from the first query's window start to the sequence's end, into
// [batch][n_kv][n][d]; else rows pos[b] + t into [batch][n][n_kv][d].
template <bool F32, bool EXPAND>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const Q4Rows p) {
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y;
    // EXPAND: blockIdx.z is (K / V, KV head), so that a thread's rows follow without a division
    const int which = EXPAND ? blockIdx.z / p.c.n_kv : blockIdx.z;
    const int head = EXPAND ? blockIdx.z - which * p.c.n_kv : 0;
    const int upr_log2 = p.d_log2 - 3;
    long long first;
    uint32_t rows = (uint32_t)p.n;
    bool bad = false;
    if (EXPAND) {
        const int len = p.seq_lens[b];
        bad = len < p.n_tok || (!p.c.ring && len > p.c.cap) || len > p.max_seq_len;
        first = p.window ? max(0, len - p.n_tok - p.window + 1) : 0;
        if (blockIdx.x == 0 && threadIdx.x == 0 && blockIdx.z == 0)
            p.lens_out[b] = bad ? 0 : (int)(len - first);
        if (bad) return;  // reported by the attention launch, which sees length 0
        rows = (uint32_t)(len - first);
    } else {
        const int r0 = p.pos[b];
        bad = r0 < 0 || (!p.c.ring && (long long)r0 + p.n > p.c.cap);
        first = r0;
        if (bad && blockIdx.x == 0 && threadIdx.x == 0 && which == 0)
            report(p.err, GEMMA_DEVERR_WRITE_POS);
    }
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(which ? p.c.v_codes : p.c.k_codes);
    const uint16_t* scales =
        reinterpret_cast<const uint16_t*>(which ? p.c.v_scales : p.c.k_scales);
    const uint32_t units = (EXPAND ? rows : rows * (uint32_t)p.c.n_kv) << upr_log2;
    const size_t out0 = EXPAND ? ((size_t)b * p.c.n_kv + head) * (size_t)p.n
                               : (size_t)b * p.n * p.c.n_kv;
    for (uint32_t base = blockIdx.x * (kThreads * kAhead) + threadIdx.x; base < units;
         base += gridDim.x * (kThreads * kAhead)) {
        uint32_t word[kAhead], sc[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const uint32_t unit = base + a * kThreads;
            const uint32_t row_in = unit >> upr_log2, u = unit & ((1u << upr_log2) - 1);
            word[a] = sc[a] = 0;
            if (unit >= units || bad) continue;
            uint32_t t = row_in, h = head;
            if (!EXPAND) p.split(row_in, t, h);
            size_t row;
            if (q4_row(p.c, b, (int)h, first + t, row)) {
                word[a] = codes[(row << upr_log2) + u];
                sc[a] = scales[(row << (upr_log2 - 3)) + (u >> 3)];
            } else if (u == 0 && h == 0) {
                report(p.err, GEMMA_DEVERR_PAGE);
            }
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const uint32_t unit = base + a * kThreads;
            if (unit < units)
                q4_store<F32>(p.dst[which], ((out0 << upr_log2) + unit) * 8, word[a], sc[a]);
        }
    }
}

int log2_of(int d) {
    int l = 0;
    while ((1 << l) < d) ++l;
    return l;
}

// grid of one launch over (units of a sequence, sequence, K / V): about sixteen CTAs per SM at most
dim3 q4_grid(long long rows, int n_kv, int head_dim, long long batch, bool two, int n_sm) {
    const long long units = rows * n_kv * (head_dim / 8), work = kThreads * kAhead;
    const long long blocks = (units + work - 1) / work;
    long long limit = (long long)n_sm * 16 / (batch * (two ? 2 : 1));
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
    p.kv_log2 = (c.n_kv & (c.n_kv - 1)) ? -1 : log2_of(c.n_kv);
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
    p.kv_log2 = (c.n_kv & (c.n_kv - 1)) ? -1 : log2_of(c.n_kv);
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
    p.kv_log2 = (c.n_kv & (c.n_kv - 1)) ? -1 : log2_of(c.n_kv);
    p.seq_lens = seq_lens;
    p.lens_out = lens_out;
    p.n_tok = n_tok;
    p.max_seq_len = max_seq_len;
    p.window = window;
    dim3 grid = q4_grid(slots, 1, head_dim, (long long)batch * c.n_kv, c.v_codes != nullptr, n_sm);
    grid.y = (unsigned)batch;
    grid.z *= (unsigned)c.n_kv;
    return launch_pdl(q4_read_kernel<false, true>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace gemma
