// sample.cu -- one token per row of logits by temperature, top-k, top-p and min-p.
//
// Per row, with z = softcap * tanh(x / softcap) (x without a cap) and the candidates (neither NaN
// nor -inf) in the order of falling x, equal ones by index:
//   keep the first top_k;  w = exp((z - z_max) / T);  keep the shortest prefix whose weights sum to
//   at least top_p of the kept ones' sum;  keep those with w >= min_p;  draw the first whose
//   running sum exceeds u times the sum of what is kept.
//
// No sort: the order of a row is a count per distinct value. bf16 has 65,536 of them, so one pass
// over the logits fills a histogram in shared memory (16-bit counters, 128 KB; the row's slices
// go to the CTAs of a cluster, at most 65,535 logits each, whose counts meet through distributed
// shared memory), and everything else works on counts and on at most a few thousand weights, each
// evaluated once in pairs of fp32 numbers (2^-40): cuts and draws fall between the same tokens as in
// a 64-bit evaluation of the definition. Ties inside a value are a division, and one look at the
// slice that holds the wanted occurrence finds its index. fp32 logits take the same histogram over
// their upper 16 bits, whose bins' weights are summed into global memory as integers (43 bits below
// the bin's own largest weight, so the order of the additions does not matter). The few hundred
// logits of a bin that a cut or the draw falls into are gathered and put in order; a bin of more
// than 1,024 takes the histogram again, over its lower 16 bits (a row of 262,144, flat
// and with a cap: 81 us, 190 with histograms of the bins; half of it are the weights, not their
// atomics: with sums in shared memory it took 9 us longer).
//
// Rows with a top_k of at most 256 (and fp32 rows without one or a cap) hardly get there: a launch
// ahead (list_kernel) draws them from the list of their largest logits, and flags those that it
// could not decide.
//
// What bounds it, per row of 262,144 bf16 logits (0.08 us at the memory's rate): latencies. One row with
// top_k 64: 14.5 us, of it 2.5 for reading the slices and the rest barriers of the cluster, the
// list's order and two launches; a row by histogram: 29 us, of it 3
// for counting (bound by shared-memory atomics; runs of eight equal logits count as one, so that
// a row masked with one finite value does not queue on one counter), 4.5 for merging the counts,
// 12 for cuts and draw. 64 rows by histogram: 106 us (three rounds of clusters), of which 5 us
// would do at the memory's rate.
#include <atomic>

#include <cuda_bf16.h>

#include "common.cuh"
#include "sample.h"

namespace gemma {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 65536, kGroups = 2048;  // 32 bins per group
constexpr int kMaxCtas = 16;
constexpr uint32_t kListK = 256;  // longest short list
// what a row costs one CTA, or a cluster, besides counting its slice: in logits of the slice
constexpr double kAloneCost = 140e3, kClusterCost = 95e3;
constexpr uint32_t kGather = kThreads;  // fp32: numbers of one upper half that are put in order

// Order-preserving key of a number (-0 as +0), its inverse, and the candidates' range of keys:
// above -inf, not above +inf.
template <bool F32>
struct Key;
template <>
struct Key<false> {
    static constexpr uint32_t kLow = 0x0080u, kInf = 0xff80u;
    __device__ static uint32_t of(uint32_t u) {
        if ((u & 0x7fffu) == 0) u = 0;
        return u & 0x8000u ? ~u & 0xffffu : u | 0x8000u;
    }
    __device__ static float value(uint32_t key) {
        const uint32_t u = key & 0x8000u ? key & 0x7fffu : ~key & 0xffffu;
        return __uint_as_float(u << 16);
    }
};
template <>
struct Key<true> {
    static constexpr uint32_t kLow = 0x00800000u, kInf = 0xff800000u;
    __device__ static uint32_t of(uint32_t u) {
        if ((u & 0x7fffffffu) == 0) u = 0;
        return u & 0x80000000u ? ~u : u | 0x80000000u;
    }
    __device__ static float value(uint32_t key) {
        return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
    }
};

__device__ __forceinline__ uint32_t peer_addr(const void* local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(r)
                 : "r"(smem_u32(local)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ld_peer(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
// Barrier of the row's CTAs, ordering their shared memory.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Unevaluated sums h + l of two fp32 numbers, |l| at most half a unit of h (Dekker's and Knuth's
// error-free sums and products). Every operation is an intrinsic: contracted or reordered they
// would lose their error terms.
struct F2 {
    float h, l;
};
__device__ __forceinline__ F2 fast_sum(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return F2{s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ F2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    return F2{s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
// (sums and products drop the products of two error terms: an error of a few 2^-47 of the larger
// operand, so a difference keeps the operands' absolute accuracy)
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    const F2 s = two_sum(a.h, b.h);
    return fast_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ F2 operator+(float a, F2 b) {  // |a| >= |b|
    const F2 s = fast_sum(a, b.h);
    return fast_sum(s.h, __fadd_rn(s.l, b.l));
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    const float m = __fmul_rn(a.h, b.h);
    float e = __fmaf_rn(a.h, b.h, -m);
    e = __fmaf_rn(a.h, b.l, e);
    return fast_sum(m, __fmaf_rn(a.l, b.h, e));
}
__device__ __forceinline__ F2 operator/(F2 a, F2 b) {
    // a first quotient from an approximate reciprocal, and one correction of what it leaves
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b.h));
    const float q = __fmul_rn(a.h, r);
    const float d = __fadd_rn(__fmaf_rn(-q, b.h, a.h), __fmaf_rn(-q, b.l, a.l));
    return fast_sum(q, __fmul_rn(d, r));
}

// 2^(i / 64) as such sums.
__constant__ float2 c_exp2[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f},
    {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f},
    {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f},
    {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f},
    {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f},
    {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f},
    {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f},
    {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f},
    {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f},
    {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f},
    {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f},
    {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f}};

// e^x = t (1 + e1) for -60 < x <= 0: x = (64 k + i) ln 2 / 64 + r with |r| < 0.0055, t = 2^k 2^(i/64)
// and e1 = e^r - 1 by its series, whose first terms keep their error terms (the fifth is below 2^-46).
__device__ __forceinline__ void exp_parts(F2 x, const float2* exp2, F2& t, F2& e1) {
    const float n = rintf(x.h * 92.332482616893656f);  // 64 / ln 2
    // ln 2 / 64 in four parts of 11 bits and a rest (n has at most 13: the products are exact)
    const F2 nb = two_sum(__fmul_rn(n, -0x1.2140000000000p-18f), __fmul_rn(n, -0x1.fbc0000000000p-29f));
    const F2 r = (x + F2{__fmul_rn(n, -0x1.62c0000000000p-7f), 0.f}) + fast_sum(nb.h, __fadd_rn(nb.l, __fmul_rn(n, -0x1.473de60000000p-40f)));
    const F2 r2 = r * r;
    const float c = r.h * r2.h * (0.16666667f + r.h * (0.041666668f + r.h * 0.0083333333f));
    e1 = r + (F2{0.5f * r2.h, 0.5f * r2.l} + F2{c, 0.f});
    const int k = (int)n;
    const float2 f = exp2[k & 63];
    const float sc = __uint_as_float((uint32_t)(127 + (k >> 6)) << 23);
    t = F2{f.x * sc, f.y * sc};
}
// e^x for x <= 0. Below -60: 0.
__device__ __forceinline__ F2 exp_f2_here(F2 x, const float2* exp2) {
    if (!(x.h > -60.f)) return F2{0.f, 0.f};
    F2 t, e1;
    exp_parts(x, exp2, t, e1);
    return (1.f + e1) * t;
}
// e^x - 1 for x <= 0, small ones (t = 1) to full relative accuracy.
__device__ __forceinline__ F2 expm1_f2_here(F2 x, const float2* exp2) {
    if (!(x.h > -60.f)) return F2{-1.f, 0.f};
    F2 t, e1;
    exp_parts(x, exp2, t, e1);
    return (-1.f + t) + t * e1;
}

// One copy of each, for the many places that need it once: a row's steps run one after another, and
// code that is fetched for a single use costs more than the call (9 fp32 rows 31.7 -> 29.7 us).
__device__ __noinline__ F2 exp_f2(F2 x, const float2* exp2) { return exp_f2_here(x, exp2); }
__device__ __noinline__ F2 expm1_f2(F2 x, const float2* exp2) { return expm1_f2_here(x, exp2); }

// A place in a row's order: the tokens above key `key`, and of key itself the first `ties`.
struct Cut {
    uint32_t key;
    uint32_t ties;
};

typedef unsigned long long u64;

struct Shared {
    uint32_t count[kGroups];  // candidates per group of 32 bins
    // weights per group, and then their running sums from the highest group down (place d: group
    // kGroups - 1 - d), inclusive; fp32: the same over the lower halves of one upper half
    u64 before[kGroups], before2[kGroups];
    float2 exp2[64];
    uint32_t mine[kGroups / 32], any[kGroups / 32];  // groups with counts: this CTA's, the row's
    uint32_t live[kGroups / 32];                     // the row's, of whole numbers or upper halves
    uint32_t open[kWarps];
    int row;
    u64 part[kWarps];
    uint32_t upart[kWarps];
    int top[kWarps];
    uint32_t found, key, n;
    u64 m, start;
    uint32_t own_max, index, listed[2], queued[2];  // fp32, see gather and the weights' sums
    uint16_t rank[kGather];
};

// A CTA's slice of a row's logits, and the row's weights. T threads.
template <bool F32, int T>
struct Slice {
    const SampleParams& p;
    const float2* exp2;  // shared copy of c_exp2
    u64* part;           // shared, one per warp
    int C, rank, row;
    long long i0, i1;
    // 1 / (t_scale T), the largest t_scale z, -2 / (scale softcap)
    F2 inv_t, zmax, inner;
    float t_scale, scale;
    uint32_t key_max;    // key of the row's largest candidate
    int tid, warp, lane;

    using K = Key<F32>;

    __device__ Slice(const SampleParams& p_, float2* exp2_, u64* part_, int C_)
        : p(p_), exp2(exp2_), part(part_), C(C_) {
        tid = threadIdx.x;
        warp = tid >> 5;
        lane = tid & 31;
        row = blockIdx.x / C;
        rank = blockIdx.x - row * C;
        const long long per = (p.vocab + C - 1) / C;
        i0 = min((long long)rank * per, (long long)p.vocab);
        i1 = min(i0 + per, (long long)p.vocab);
        scale = p.softcap > 1.f ? 0x1p-32f : 1.f;
        inner = p.softcap > 0.f ? F2{-2.f, 0.f} / F2{p.softcap * scale, 0.f} : F2{0.f, 0.f};
        for (int i = tid; i < 64; i += T) exp2_[i] = c_exp2[i];
    }

    // t_scale z of a logit, z = x or c tanh(x / c) = -+c m / (2 + m), m = exp(-2 |x| / c) - 1: with 1 - exp() a cap far
    // above the logits would cancel their digits. Below |x| / c = 2^-25 it is x to 2^-50. (scale keeps
    // 2 / c and |x| / c in range for the largest caps.)
    template <bool HERE = false>  // (for loops over all logits)
    __device__ __forceinline__ F2 capped(float x) const {
        if (!(p.softcap > 0.f)) return F2{x * t_scale, 0.f};
        const F2 y = F2{fabsf(x) * scale, 0.f} * inner;
        if (y.h > -0x1p-24f) return F2{x * t_scale, 0.f};
        const F2 m = HERE ? expm1_f2_here(y, exp2) : expm1_f2(y, exp2);
        F2 t = F2{-m.h, -m.l} / (2.f + m);
        if (isinf(x)) t = F2{1.f, 0.f};
        t = t * F2{p.softcap * t_scale, 0.f};
        return x < 0.f ? F2{-t.h, -t.l} : t;
    }
    // Above 2^64 a temperature and the z that it divides are taken 2^-64 times: 1 / T and the
    // differences of the largest logits would leave fp32's range.
    __device__ void set_temperature(float t) {
        t_scale = t > 0x1p64f ? 0x1p-64f : 1.f;
        inv_t = t > 0.f ? F2{1.f, 0.f} / F2{t * t_scale, 0.f} : F2{0.f, 0.f};
    }
    // exp((z - top) / T) of a logit z <= top, both times t_scale
    template <bool HERE = false>
    __device__ __forceinline__ F2 relative(F2 z, F2 top) const {
        if (isinf(top.h)) return F2{isinf(z.h) && z.h > 0.f ? 1.f : 0.f, 0.f};
        const F2 d = z + F2{-top.h, -top.l};
        if (d.h == 0.f) return F2{1.f, 0.f};
        if (!(d.h > -1e30f)) return F2{0.f, 0.f};
        return HERE ? exp_f2_here(d * inv_t, exp2) : exp_f2(d * inv_t, exp2);
    }
    __device__ F2 weight(uint32_t key) const {
        return key == key_max ? F2{1.f, 0.f} : relative(capped(K::value(key)), zmax);
    }
    // Most of a row lies below e^-9 / vocab of the largest weight: single precision is enough there
    // (the rounding of all of them together is within 2^-34 of the largest; without a cap). Adds such a
    // weight, exp(d) with d < below, to `tiny`, else returns false.
    __device__ bool tiny_weight(uint32_t key, float below, float& tiny) const {
        if (key == key_max || isinf(zmax.h)) return false;
        // (zmax.l is zero without a cap)
        const F2 a = two_sum(K::value(key) * t_scale, -zmax.h);
        const float d = __fmul_rn(a.h, inv_t.h);
        if (!(d < below)) return false;
        const float rest = __fmaf_rn(a.h, inv_t.h, -d) + (a.l * inv_t.h + a.h * inv_t.l);
        if (d > -80.f) tiny += expf(d) * (1.f + rest);
        return true;
    }
    // n weights in units of 2^-43, rounded
    __device__ u64 units(F2 w, uint32_t n) const {
        if (!(w.h > 0.f)) return 0;
        const F2 m = w * F2{(float)n, 0.f};  // n < 2^24: exact
        return (u64)(__float2ll_rn(m.h * 0x1p43f) + __float2ll_rn(m.l * 0x1p43f));
    }

    // Calls vec for every aligned 16 bytes of the slice and one for the elements around them.
    template <class V, class O>
    __device__ void for_slice(V vec, O one) {
        for_slice_at([&](uint4 v, long long) { vec(v); }, [&](uint32_t u, long long) { one(u); });
    }
    // The same, with the (first) element's index in the row.
    template <class V, class O>
    __device__ void for_slice_at(V vec, O one) {
        constexpr int E = F32 ? 4 : 8;
        const long long base = (long long)row * p.vocab;
        const long long b0 = base + i0, b1 = base + i1;
        const long long a0 = min((b0 + E - 1) / E * E, b1), a1 = max(b1 / E * E, a0);
        auto load1 = [&](long long i) -> uint32_t {
            return F32 ? static_cast<const uint32_t*>(p.logits)[i]
                       : static_cast<const uint16_t*>(p.logits)[i];
        };
        for (long long i = b0 + tid; i < a0; i += T) one(load1(i), i - base);
        const uint4* v = reinterpret_cast<const uint4*>(p.logits) + a0 / E;
        const int n = (int)((a1 - a0) / E);
        int i = tid;
        for (; i + 3 * T < n; i += 4 * T) {
            uint4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = v[i + k * T];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                vec(x[k], a0 - base + (long long)(i + k * T) * E);
        }
        for (; i < n; i += T) vec(v[i], a0 - base + (long long)i * E);
        for (long long j = a1 + tid; j < b1; j += T) one(load1(j), j - base);
    }

    // Calls take(bits, index) for the few elements whose key is wanted. bf16: where the largest of
    // eight is; fp32: from one copy of it for four elements (instructions fetched for a rare use
    // hold up the other warps).
    template <class W, class F>
    __device__ void for_wanted(W wanted, F take) {
        for_slice_at([&](uint4 v, long long at) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (!F32) {
                if (!wanted(K::of(vec_max(v)))) return;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t bits = w[e / 2] >> 16 * (e & 1) & 0xffffu;
                    if (wanted(K::of(bits))) take(bits, at + e);
                }
                return;
            }
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) hits |= (uint32_t)wanted(K::of(w[e])) << e;
            while (hits) {
                const int e = __ffs(hits) - 1;
                hits &= hits - 1;
                take(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w, at + e);
            }
        }, [&](uint32_t bits, long long at) {
            if (wanted(K::of(bits))) take(bits, at);
        });
    }

    // The largest key of this thread's part of the slice (0 if it has no candidate).
    __device__ uint32_t thread_max() {
        uint32_t best = 0;
        for_slice([&](uint4 v) {
            uint32_t m;
            if (F32) {
                m = __float_as_uint(fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                                          fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))));
            } else {
                m = vec_max(v);
            }
            m = K::of(m);
            if (m <= K::kInf) best = max(best, m);
        }, [&](uint32_t u) {
            const uint32_t key = K::of(u);
            if (key <= K::kInf) best = max(best, key);
        });
        return best >= K::kLow ? best : 0;
    }
    // Largest of eight bf16 (NaN only if all are), as bits.
    __device__ static uint32_t vec_max(const uint4& v) {
        uint32_t m;
        asm("{\n\t.reg .b32 a, b;\n\tmax.bf16x2 a, %1, %2;\n\tmax.bf16x2 b, %3, %4;\n\t"
            "max.bf16x2 %0, a, b;\n\t}"
            : "=r"(m)
            : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
        const float f = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        return __float_as_uint(f) >> 16;
    }
    // How many of the n distinct entries are larger than entry i0 + tid / 4, which is e: four lanes
    // share an entry.
    __device__ uint32_t larger(const u64* entries, uint32_t n, uint32_t i0, u64& e) const {
        const uint32_t i = i0 + tid / 4, q = (n + 3) / 4 | 1u;  // (odd: the lanes' reads in other banks)
        e = entries[min(i, n - 1)];
        uint32_t count = 0;
        const uint32_t j1 = min((tid & 3) * q + q, n);
#pragma unroll 4
        for (uint32_t j = (tid & 3) * q; j < j1; ++j) count += entries[j] > e;
        count += __shfl_xor_sync(0xffffffffu, count, 1);
        return count + __shfl_xor_sync(0xffffffffu, count, 2);
    }
    // Inclusive sums over the warp's lanes.
    template <class N>
    __device__ N warp_sums(N x) const {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const N y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    }
    // Sum of the values of the CTA's threads before this one.
    template <class N>
    __device__ N sum_before(N v) {
        const N x = warp_sums(v);
        __syncthreads();  // (`part` may still be read)
        if (lane == 31) part[warp] = x;
        __syncthreads();
        const N all = warp_sums(lane < T / 32 ? (N)part[lane] : (N)0);
        const N base = __shfl_sync(0xffffffffu, all, (warp + 31) & 31);
        return (warp ? base : (N)0) + x - v;
    }
};

// The parameters of a row; false if they are out of range.
struct Filters {
    float t, top_p, min_p, u;
    int top_k;
    __device__ bool load(const SampleParams& p, int row) {
        t = p.temperature ? p.temperature[row] : 1.f;
        top_k = p.top_k ? p.top_k[row] : 0;
        top_p = p.top_p ? p.top_p[row] : 1.f;
        min_p = p.min_p ? p.min_p[row] : 0.f;
        u = p.uniform[row];
        return t >= 0.f && isfinite(t) && top_p == top_p && min_p == min_p && u >= 0.f && u < 1.f;
    }
    // How many of the largest logits draw the row: one, or top_k; 0: it has no such number.
    __device__ uint32_t want() const {
        return t == 0.f ? 1u : top_k > 0 ? (uint32_t)top_k : 0u;
    }
    // Whether the short list below takes the row on.
    template <bool F32>
    __device__ bool listed(float softcap) const {
        const uint32_t n = want();
        return n ? n <= kListK : F32 && !(softcap > 0.f);
    }
};

// The short list. A row with a top_k up to kListK, and an fp32 row without one or a cap, is drawn
// from its n = top_k (kListK) largest logits alone. In us, the list and the histograms: bf16, one
// row of 262,144: top_k 20 12.9, 27.8; 256 21.6, 24.7; 64 rows: 35.2, 104.8 and 55.0, 94.8; fp32, 9
// rows of 70,001 that top_p 0.9 ends within the list: 29.2, 46. (With a cap the sum of all weights
// took longer than the histograms do: 157, 88.) The n-th largest of a CTA's threads' largest keys bounds
// the row's n-th largest logit from below, and so does the smallest over the CTAs of each one's
// (n / C)-th: every CTA sends its slice's keys down to the higher of these bounds to one of them,
// which orders them and walks down their running weights. Without a top_k the sum of all weights is
// needed too (one evaluation per logit), and the draw may lie beyond the list; lists may also be too
// long (many equal logits): such rows are left to the kernel below, as are all others.
constexpr int kListThreads = 256;
constexpr uint32_t kListMax = 1024, kListSpace = 2048;

struct ListShared {
    float2 exp2[64];
    u64 part[kListThreads / 32];
    uint32_t upart[kListThreads / 32];
    uint32_t bound[2], largest, n_list, n_near;
    // the leading CTA's: entries and weight of each slice, the entries, and in order
    uint32_t counts[kMaxCtas];
    u64 sums[kMaxCtas];
    u64 all;
    alignas(16) u64 pool[kListMax];  // (also the threads' largest keys, read 16 bytes at a time)
    u64 order[kListK], space[kListSpace];
};
static_assert(offsetof(ListShared, pool) % 16 == 0, "read 16 bytes at a time");

template <bool F32>
__global__ void __launch_bounds__(kListThreads) list_kernel(const SampleParams p, int C) {
    pdl_launch_dependents();
    constexpr int T = kListThreads;
    using K = Key<F32>;
    extern __shared__ __align__(16) uint8_t smem[];
    ListShared& s = *reinterpret_cast<ListShared*>(smem);
    pdl_wait();
    Slice<F32, T> r(p, s.exp2, s.part, C);
    const int tid = r.tid, warp = r.warp, lane = r.lane, row = r.row, rank = r.rank;
    const int lead = row % C;  // (the rows' leaders on different SMs: CTAs of a rank tend to share one)
    Filters f;
    const bool good = f.load(p, row);
    const uint32_t want = f.want();
    // (the same in every CTA of the row)
    if (!good || !f.listed<F32>(p.softcap)) {
        if (rank == lead && tid == 0) {
            p.open[row] = good;
            if (!good) {
                p.token[row] = -1;
                report(p.err, GEMMA_DEVERR_SAMPLE);
            }
        }
        return;
    }
    const uint32_t n = want ? want : kListK;
    r.set_temperature(f.t);
    const uint32_t best = r.thread_max();

    // The n-th and the (n / C)-th largest of the threads' keys (0 if fewer threads have one): every
    // thread counts the larger ones; the thread's number makes them distinct (fp32: in place of the
    // key's lowest bits, which makes the bound a little lower).
    uint32_t* tops = reinterpret_cast<uint32_t*>(s.pool);
    const uint32_t bound = F32 ? best & ~0xffu : best;
    const uint32_t mine = (F32 ? bound : best << 8) | (T - 1 - tid);
    tops[tid] = mine;
    const uint32_t mx = __reduce_max_sync(0xffffffffu, best);
    if (lane == 0) s.upart[warp] = mx;
    __syncthreads();
    uint32_t above = 0;
#pragma unroll 8
    for (int k = 0; k < T / 4; ++k) {
        const uint4 v = reinterpret_cast<const uint4*>(tops)[k];
        above += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
    }
    if (above == n - 1) s.bound[0] = bound;
    if (above == (n + C - 1) / C - 1) s.bound[1] = bound;
    if (warp == 0) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, lane < T / 32 ? s.upart[lane] : 0u);
        if (lane == 0) {
            s.largest = m;
            s.n_list = s.n_near = 0;
        }
    }
    cluster_barrier();
    uint32_t lg = 0, high = 0, low = 0xffffffffu;
    if (lane < C) {
        high = ld_peer(peer_addr(&s.bound[0], lane));
        low = ld_peer(peer_addr(&s.bound[1], lane));
        lg = ld_peer(peer_addr(&s.largest, lane));
    }
    const uint32_t pivot = max(__reduce_max_sync(0xffffffffu, high),
                               __reduce_min_sync(0xffffffffu, low));
    r.key_max = __reduce_max_sync(0xffffffffu, lg);
    const uint32_t floor_key = max(pivot, K::kLow), room = kListSpace / C;
    const uint32_t space = peer_addr(s.space + rank * room, lead);
    // keys down to the bound: falling keys, then rising indices, in one number
    auto take = [&](uint32_t bits, long long at) {
        const uint32_t key = K::of(bits);
        const uint32_t i = atomicAdd(&s.n_list, 1u);
        if (i < room) st_peer(space + 8 * i, (u64)key << 32 | (0xffffffffu - (uint32_t)at));
    };
    r.for_wanted([&](uint32_t key) { return key >= floor_key && key <= K::kInf; }, take);
    const bool need_sum = F32 && !want && r.key_max;
    if (need_sum || rank == lead) r.zmax = r.capped(K::value(max(r.key_max, K::kLow)));
    if (need_sum) {
        // Equal logits round alike, and a row may have a million of them: a thread's sum is a pair of
        // fp32 numbers and is rounded once, to units of 2^-46 (a slice has fewer than 2^17 logits),
        // the CTA's to 2^-43.
        F2 mine{0.f, 0.f};
        auto add = [&](F2 w) { mine = mine + w; };
        const float below = -9.f - logf((float)p.vocab);
        // (those near the largest one, a few per hundred, are weighed together afterwards: in place
        // one lane's would hold up its warp)
        uint32_t* near = reinterpret_cast<uint32_t*>(s.pool);
        const uint32_t* x = static_cast<const uint32_t*>(p.logits) + (long long)row * p.vocab;
        const int i1 = (int)r.i1;
        auto load = [&](int i) { return i < i1 ? x[i] : 0x7fffffffu; };  // (NaN: none)
        int i0 = (int)r.i0 + tid;
        uint32_t next[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) next[k] = load(i0 + k * T);
#pragma unroll 1
        for (; i0 < i1; i0 += 4 * T) {
            uint32_t now[4];
            float tiny = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                now[k] = K::of(next[k]);
                next[k] = load(i0 + (4 + k) * T);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t key = now[k];
                if (key < K::kLow || key > K::kInf || r.tiny_weight(key, below, tiny)) continue;
                const uint32_t i = atomicAdd(&s.n_near, 1u);
                if (i < 2 * kListMax) near[i] = key;
            }
            const F2 sum = two_sum(mine.h, tiny);
            mine = F2{sum.h, __fadd_rn(mine.l, sum.l)};
        }
        __syncthreads();
        const uint32_t n_near = s.n_near;
        if (n_near <= 2 * kListMax) {
            for (uint32_t i = tid; i < n_near; i += T) add(r.weight(near[i]));
        } else {  // no room: all of them where they lie
            for (int i = (int)r.i0 + tid; i < i1; i += T) {
                const uint32_t key = K::of(load(i));
                float tiny = 0.f;  // (those are in the sum already)
                if (key >= K::kLow && key <= K::kInf && !r.tiny_weight(key, below, tiny))
                    add(r.weight(key));
            }
        }
        const u64 sum = (u64)(__float2ll_rn(mine.h * 0x1p46f) + __float2ll_rn(mine.l * 0x1p46f));
        const u64 b = r.sum_before(sum);
        if (tid == T - 1) st_peer(peer_addr(&s.sums[rank], lead), (b + sum + 4) >> 3);
    }
    __syncthreads();
    if (tid == 0) st_peer(peer_addr(&s.counts[rank], lead), s.n_list);
    cluster_barrier();
    if (rank != lead) return;  // (its shared memory is read no more)

    if (r.key_max == 0) {  // no candidate
        if (tid == 0) {
            p.open[row] = 0;
            p.token[row] = -1;
            report(p.err, GEMMA_DEVERR_SAMPLE);
        }
        return;
    }
    const uint32_t count = lane < C ? s.counts[lane] : 0u;
    const uint32_t ends = r.warp_sums(count);  // of CTA lane's entries among all
    const uint32_t total = __shfl_sync(0xffffffffu, ends, 31);
    if (__any_sync(0xffffffffu, count > room) || total > kListMax) {
        if (tid == 0) p.open[row] = 1;
        return;
    }
    for (uint32_t i0 = warp * 32; i0 < total; i0 += T) {
        const uint32_t i = i0 + lane;
        uint32_t q = 0;
        for (int c = 0; c < C; ++c) q += i >= __shfl_sync(0xffffffffu, ends, c);
        const uint32_t first = __shfl_sync(0xffffffffu, ends - count, q & 31);
        if (i < total) s.pool[i] = s.space[q * room + i - first];
    }
    __syncthreads();
    const uint32_t kept_n = min(n, total);
    for (uint32_t i0 = 0; i0 < total; i0 += T / 4) {
        u64 e;
        const uint32_t before = r.larger(s.pool, total, i0, e);
        if (!(tid & 3) && i0 + tid / 4 < total && before < kept_n) s.order[before] = e;
    }
    __syncthreads();
    const bool have = tid < (int)kept_n;
    const u64 e = have ? s.order[tid] : 0;
    const uint32_t key = (uint32_t)(e >> 32);
    const F2 w = have ? r.weight(key) : F2{0.f, 0.f};
    const u64 m = have ? r.units(w, 1u) : 0;
    const u64 run = r.sum_before(m) + m;
    u64 all;
    if (need_sum) {
        all = __shfl_sync(0xffffffffu, r.warp_sums(lane < C ? s.sums[lane] : (u64)0), 31);
    } else {
        if (tid == T - 1) s.all = run;
        __syncthreads();
        all = s.all;
    }
    auto first = [&](bool yes) {  // lowest thread that says yes, or T
        const unsigned b = __ballot_sync(0xffffffffu, yes);
        __syncthreads();
        if (lane == 0) s.upart[warp] = b ? warp * 32 + __ffs(b) - 1 : T;
        __syncthreads();
        return __reduce_min_sync(0xffffffffu, s.upart[lane & (T / 32 - 1)]);
    };
    auto run_at = [&](uint32_t i) {
        __syncthreads();
        if (tid == (int)i) s.all = run;
        __syncthreads();
        return s.all;
    };
    // how many entries are kept, and their weight
    uint32_t keep = kept_n;
    bool open = need_sum && (pivot != 0 || total > n);  // what is kept may reach beyond the list
    bool fits = true;
    u64 kept = all;
    if (f.top_p <= 0.f) {
        keep = 1;
        open = false;
        kept = run_at(0);
    } else if (f.top_p < 1.f) {
        const u64 need = min(max((u64)ceil((double)f.top_p * (double)all), (u64)1), all);
        const uint32_t i = first(have && run >= need);
        if (i < kept_n) {
            keep = i + 1;
            open = false;
            kept = run_at(i);
        } else {
            fits = false;
        }
    }
    if (f.min_p > 0.f) {
        const bool below = have && key != r.key_max &&
                           !(w.h > f.min_p || (w.h == f.min_p && w.l >= 0.f));
        const uint32_t i = first(below);
        if (i < keep) {
            keep = i;
            kept = run_at(i - 1);
            fits = true;  // (whatever top_p left undecided lies below the floor)
        } else if (open) {
            fits = false;
        }
    }
    if (fits) {
        const u64 need = min((u64)((double)f.u * (double)kept) + 1, kept);
        const uint32_t i = first(have && run >= need);
        if (i >= kept_n) fits = false;
        else if (tid == (int)i) p.token[row] = (int32_t)(0xffffffffu - (uint32_t)e);
    }
    if (tid == 0) p.open[row] = !fits;
}

template <bool F32>
struct Row : Slice<F32, kThreads> {
    using Base = Slice<F32, kThreads>;
    using K = Key<F32>;
    using Base::C; using Base::lane; using Base::p; using Base::rank; using Base::row;
    using Base::tid; using Base::warp; using Base::for_slice; using Base::warp_sums;
    using Base::sum_before;
    Shared& s;
    uint32_t* hist;   // [kBins / 2] pairs of 16-bit counters
    uint32_t* merged; // [groups of this CTA][32] counts of the whole row (more than one CTA)
    uint32_t best;    // fp32: this thread's largest candidate key

    __device__ Row(const SampleParams& p_, Shared& s_, uint32_t* hist_, int C_)
        : Base(p_, s_.exp2, s_.part, C_), s(s_), hist(hist_), merged(hist_ + kBins / 2), best(0) {}

    // Histogram of this CTA's slice. bf16: of the keys; fp32: of the keys' upper halves (level 0)
    // or of the lower halves of those with upper half `upper`.
    __device__ void count_slice(int level, uint32_t upper) {
        for (int i = tid; i < kBins / 8; i += kThreads)
            reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        auto add = [&](uint32_t u, uint32_t n) {
            const uint32_t key = K::of(u);
            if (key < K::kLow || key > K::kInf) return;
            uint32_t bin = key;
            if (F32) {
                if (level == 0) {
                    best = max(best, key);
                    bin = key >> 16;
                } else {
                    if (key >> 16 != upper) return;
                    bin = key & 0xffffu;
                }
            }
            atomicAdd(&hist[bin >> 1], n << (16 * (bin & 1)));
        };
        for_slice([&](uint4 v) {
            if (F32) {
                if (v.x == v.y && v.x == v.z && v.x == v.w) {
                    add(v.x, 4);
                } else {
                    add(v.x, 1);
                    add(v.y, 1);
                    add(v.z, 1);
                    add(v.w, 1);
                }
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                if (v.x == v.y && v.x == v.z && v.x == v.w && (v.x & 0xffffu) == v.x >> 16) {
                    add(v.x & 0xffffu, 8);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        add(w[k] & 0xffffu, 1);
                        add(w[k] >> 16, 1);
                    }
                }
            }
        }, [&](uint32_t u) { add(u, 1); });
        __syncthreads();
    }
    // The row's counts: group sums into every CTA's s.count, bins into their owner's `merged`
    // (group g belongs to CTA g % C). Needs every CTA's histogram, leaves them readable. A row's
    // values lie in a few hundred of the 2,048 groups, and a peer's shared memory gives only some
    // 16 bytes a clock: the CTAs first exchange which groups they have, and read no others.
    // fp32: the weight sums of the groups that the row has start at zero.
    __device__ void merge_counts(u64* mass = nullptr) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int g = h * kThreads + tid;
            uint32_t has = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(hist)[g * 4 + i];
                has |= v.x | v.y | v.z | v.w;
            }
            const unsigned word = __ballot_sync(0xffffffffu, has != 0);
            if (lane == 0) s.mine[h * kWarps + warp] = word;
            s.count[g] = 0;
        }
        if (tid < kGroups / 32) s.any[tid] = 0;
        cluster_barrier();
        for (int i = tid; i < kGroups / 32 * C; i += kThreads) {
            const uint32_t v = ld_peer(peer_addr(&s.mine[i & 63], i >> 6));
            if (v) atomicOr(&s.any[i & 63], v);
        }
        __syncthreads();
        for (int k = warp; rank + k * C < kGroups; k += kWarps) {
            const int g = rank + k * C, w = g * 16 + (lane & 15);
            if (!(s.any[g / 32] >> (g & 31) & 1u)) continue;
            if (mass) mass[g * 32 + lane] = 0ull;
            uint32_t lo = 0, hi = 0;
            // (all loads in flight at once: a peer's memory is a few hundred ns away)
            uint32_t v[kMaxCtas / 2];
#pragma unroll
            for (int i = 0; i < kMaxCtas / 2; ++i) {
                const int r = 2 * i + (lane >> 4);
                v[i] = r < C ? ld_peer(peer_addr(hist + w, r)) : 0u;
            }
#pragma unroll
            for (int i = 0; i < kMaxCtas / 2; ++i) {
                lo += v[i] & 0xffffu;
                hi += v[i] >> 16;
            }
            lo += __shfl_xor_sync(0xffffffffu, lo, 16);
            hi += __shfl_xor_sync(0xffffffffu, hi, 16);
            if (C > 1 && lane < 16)
                *reinterpret_cast<uint2*>(merged + k * 32 + 2 * lane) = make_uint2(lo, hi);
            const uint32_t sum = __reduce_add_sync(0xffffffffu, lane < 16 ? lo + hi : 0u);
            if (lane < C) st_peer(peer_addr(&s.count[g], lane), sum);
        }
        if (mass) __threadfence();
        cluster_barrier();
    }
    // count of bin 32 g + i (any CTA's)
    __device__ uint32_t bin_count(int g, int i) const {
        if (s.count[g] == 0) return 0;
        if (C == 1) return hist[g * 16 + (i >> 1)] >> (16 * (i & 1)) & 0xffffu;
        return ld_peer(peer_addr(merged + (g / C) * 32 + i, g % C));
    }

    // Weights per group to running sums, in place.
    __device__ void running_sums(u64* before) {
        const u64 a = before[kGroups - 1 - 2 * tid], b = before[kGroups - 2 - 2 * tid];
        const u64 base = sum_before(a + b);
        before[2 * tid] = base + a;
        before[2 * tid + 1] = base + a + b;
        __syncthreads();
    }
    // First place d (group kGroups - 1 - d) whose running sum is at least `need`, which the last is.
    __device__ int reach(const u64* before, u64 need) {
        const u64 prev = tid ? before[2 * tid - 1] : 0, a = before[2 * tid], b = before[2 * tid + 1];
        if (prev < need && need <= a) s.found = 2 * tid;
        if (a < need && need <= b) s.found = 2 * tid + 1;
        __syncthreads();
        const int d = (int)s.found;
        __syncthreads();
        return d;
    }
};

// Draw one row (every CTA of its cluster).
template <bool F32>
__device__ void draw_row(const SampleParams& p, Shared& s, uint32_t* hist, int C, int row) {
    using K = Key<F32>;
    Row<F32> r(p, s, hist, C);
    r.row = row;
    const int tid = r.tid, warp = r.warp, lane = r.lane, rank = r.rank;
    Filters f;
    if (!f.load(p, row)) {  // the same in every CTA of the row
        if (rank == 0 && tid == 0) {
            p.token[row] = -1;
            report(p.err, GEMMA_DEVERR_SAMPLE);
        }
        return;
    }
    const float t = f.t, top_p = f.top_p, min_p = f.min_p, u = f.u;
    const int want_k = f.top_k;
    r.set_temperature(f.t);
    s.before[tid] = s.before[tid + kThreads] = 0;
    u64* mass = F32 ? p.mass + (size_t)row * kBins : nullptr;

    r.count_slice(0, 0);
    if (F32) {
        const uint32_t mx = __reduce_max_sync(0xffffffffu, r.best);
        if (lane == 0) s.upart[warp] = mx;
        __syncthreads();
        if (warp == 0) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, s.upart[lane]);
            if (lane == 0) s.own_max = m;
        }
    }
    r.merge_counts(mass);

    // the largest candidate and the number of them
    uint32_t total = 0;
    int top = -1;
    {
        const uint32_t a = s.count[2 * tid], b = s.count[2 * tid + 1];
        const uint32_t sum = __reduce_add_sync(0xffffffffu, a + b);
        if (tid < kGroups / 32) s.live[tid] = s.any[tid];
        const int hi = __reduce_max_sync(0xffffffffu, b ? 2 * tid + 1 : a ? 2 * tid : -1);
        if (lane == 0) {
            s.upart[warp] = sum;
            s.top[warp] = hi;
        }
        __syncthreads();
        total = __reduce_add_sync(0xffffffffu, s.upart[lane]);
        top = __reduce_max_sync(0xffffffffu, s.top[lane]);
        __syncthreads();
    }
    if (total == 0) {
        if (rank == 0 && tid == 0) {
            p.token[row] = -1;
            report(p.err, GEMMA_DEVERR_SAMPLE);
        }
        cluster_barrier();  // no CTA leaves while another reads its counts
        return;
    }
    auto top_bin = [&](int g) {  // highest bin with a candidate of group g
        const unsigned any = __ballot_sync(0xffffffffu, r.bin_count(g, lane) != 0);
        return (uint32_t)(g * 32 + 31 - __clz(any));
    };
    const uint32_t bin_max = top_bin(top);

    // fp32: bins over the lower halves of the numbers with upper half `upper` (s.count and
    // `merged` then hold these)
    uint32_t at = 0xffffffffu;  // that upper half
    auto refine = [&](uint32_t upper) {
        if (at == upper) return;
        cluster_barrier();  // (peers may still read the counts)
        s.before2[tid] = s.before2[tid + kThreads] = 0;
        r.count_slice(1, upper);
        r.merge_counts();
        at = upper;
    };
    uint32_t key_max = bin_max;
    const bool greedy = t == 0.f || want_k == 1;
    const uint32_t k = want_k > 0 && (uint32_t)want_k < total ? (uint32_t)want_k : total;

    // the n-th candidate from the highest down, by counts
    auto kth = [&](uint32_t n, uint32_t& bin, uint32_t& ties) {
        const uint32_t a = s.count[kGroups - 1 - 2 * tid], b = s.count[kGroups - 2 - 2 * tid];
        const uint32_t ex = r.sum_before(a + b);
        if (ex < n && ex + a >= n) {
            s.key = kGroups - 1 - 2 * tid;
            s.n = n - ex;
        } else if (ex + a < n && ex + a + b >= n) {
            s.key = kGroups - 2 - 2 * tid;
            s.n = n - ex - a;
        }
        __syncthreads();
        const int g = (int)s.key;
        const uint32_t left = s.n;
        __syncthreads();
        const uint32_t c = r.bin_count(g, 31 - lane), y = r.warp_sums(c);
        const int l = __ffs(__ballot_sync(0xffffffffu, y >= left)) - 1;
        bin = (uint32_t)(g * 32 + 31 - l);
        ties = left - __shfl_sync(0xffffffffu, y - c, l);
    };

    Cut cut{0u, 0u};       // kept so far: this and above
    bool cut_all = true;   // or every candidate

    // fp32: the numbers with upper half `upper`, at most kGather, in the order, one per thread (the
    // same in every CTA). The CTAs exchange their slices' ones as the lower half and the place in
    // the slice; a list is written again two calls later, behind a barrier that all pass having
    // read it.
    struct Entry {
        uint32_t key, tie, index;
        bool have;
    };
    int buf = 0;
    auto gather = [&](uint32_t upper) {
        uint32_t* list = reinterpret_cast<uint32_t*>(s.before2) + buf * kGather;
        u64* pool = s.before2 + kGather;
        const uint32_t per = (uint32_t)((p.vocab + C - 1) / C);
        if (tid == 0) s.listed[buf] = 0;
        __syncthreads();
        r.for_wanted(
            [&](uint32_t key) { return key >> 16 == upper && key >= K::kLow && key <= K::kInf; },
            [&](uint32_t bits, long long at) {
                const uint32_t i = atomicAdd(&s.listed[buf], 1u);
                if (i < kGather) list[i] = K::of(bits) << 16 | (0xffffu - (uint32_t)(at - r.i0));
            });
        cluster_barrier();
        const uint32_t count = lane < C ? ld_peer(peer_addr(&s.listed[buf], lane)) : 0u;
        const uint32_t ends = r.warp_sums(count);
        const uint32_t n = min(__shfl_sync(0xffffffffu, ends, 31), kGather);
        Entry e{0u, 0u, 0u, (uint32_t)tid < n};
        uint32_t q = 0;
        for (int c = 0; c < C; ++c) q += (uint32_t)tid >= __shfl_sync(0xffffffffu, ends, c);
        const uint32_t first = __shfl_sync(0xffffffffu, ends - count, q & 31);
        u64 x = 0;
        if (e.have) {
            const uint32_t v = ld_peer(peer_addr(list + tid - first, q));
            x = (u64)(v >> 16) << 32 | (0xffffffffu - (q * per + 0xffffu - (v & 0xffffu)));
            pool[tid] = x;
        }
        __syncthreads();
        for (uint32_t i0 = 0; i0 < n; i0 += kThreads / 4) {
            u64 y;
            const uint32_t before = r.larger(pool, n, i0, y);
            if (!(tid & 3) && i0 + tid / 4 < n) s.rank[i0 + tid / 4] = (uint16_t)before;
        }
        __syncthreads();
        if (e.have) pool[s.rank[tid]] = x;
        __syncthreads();
        if (e.have) {
            x = pool[tid];
            e.key = upper << 16 | (uint32_t)(x >> 32);
            e.index = 0xffffffffu - (uint32_t)x;
        }
        // equal ones before it: from the last place where the key changes
        const bool head = e.have && (tid == 0 || (uint32_t)(pool[tid - 1] >> 32) != (uint32_t)(x >> 32));
        const unsigned heads = __ballot_sync(0xffffffffu, head);
        if (lane == 0) s.top[warp] = heads ? warp * 32 + 31 - __clz(heads) : -1;
        __syncthreads();
        const unsigned low = heads & (0xffffffffu >> (31 - lane));
        const int past = __reduce_max_sync(0xffffffffu, lane < warp ? s.top[lane] : -1);
        e.tie = tid - (low ? warp * 32 + 31 - __clz(low) : past);
        buf ^= 1;
        return e;
    };
    // whether the counts at hand are of upper halves and `bin` holds few enough numbers
    auto gathers = [&](uint32_t bin) {
        return F32 && at == 0xffffffffu && r.bin_count((int)(bin / 32), (int)(bin % 32)) <= kGather;
    };
    uint32_t drawn = 0xffffffffu;  // fp32: the index drawn, if a gathered list gave it
    if (F32)
        key_max = __reduce_max_sync(0xffffffffu,
                                    lane < C ? ld_peer(peer_addr(&s.own_max, lane)) : 0u);
    r.key_max = key_max;
    r.zmax = r.capped(K::value(key_max));

    uint32_t draw_key = key_max, draw_tie = 0;
    if (!greedy) {
        uint32_t cut_bin = 0;
        u64 cut_mass = 0;  // fp32: kept weight of the cut's own bin
        if (k < total) {
            kth(k, cut_bin, cut.ties);
            cut.key = cut_bin;
            cut_all = false;
            if (F32) {
                const uint32_t n = cut.ties;
                if (gathers(cut_bin)) {
                    const Entry e = gather(cut_bin);
                    const u64 m = (uint32_t)tid < n ? r.units(r.weight(e.key), 1u) : 0;
                    const u64 run = r.sum_before(m) + m;
                    if ((uint32_t)tid == n - 1) {
                        s.key = e.key;
                        s.n = e.tie + 1;
                        s.m = run;
                    }
                    __syncthreads();
                    cut = Cut{s.key, s.n};
                    cut_mass = s.m;
                    __syncthreads();
                } else {
                    uint32_t low;
                    refine(cut_bin);
                    kth(n, low, cut.ties);
                    cut.key = cut_bin << 16 | low;
                }
            }
        }
        // tokens of a key that are kept so far, of the c there are
        auto kept_of = [&](uint32_t key, uint32_t c) {
            return cut_all || key > cut.key ? c : key == cut.key ? min(c, cut.ties) : 0u;
        };
        auto stays = [&](const Entry& e) {
            return cut_all || e.key > cut.key || (e.key == cut.key && e.tie < cut.ties);
        };
        // fp32: weights over the lower halves of `at`, of what is kept so far
        uint32_t lower_of = 0xffffffffu;
        auto lower_masses = [&](uint32_t upper) {
            if (lower_of == upper) return;
            if (at == upper) {  // counted, but the sums gave way to the queue below
                s.before2[tid] = s.before2[tid + kThreads] = 0;
                cluster_barrier();
            }
            refine(upper);
            for (int q = warp; rank + q * C < kGroups; q += kWarps) {
                const int g = rank + q * C;
                if (s.count[g] == 0) continue;
                const uint32_t key = upper << 16 | (uint32_t)(g * 32 + lane);
                const uint32_t n = kept_of(key, r.bin_count(g, lane));
                u64 m = n ? r.units(r.weight(key), n) : 0;
                m = __shfl_sync(0xffffffffu, r.warp_sums(m), 31);
                if (lane < C) st_peer(peer_addr(&s.before2[g], lane), m);
            }
            cluster_barrier();
            r.running_sums(s.before2);
            lower_of = upper;
        };
        if (F32 && !cut_all && at == cut_bin) {
            lower_masses(cut_bin);
            cut_mass = s.before2[kGroups - 1];
        }
        if (F32) {
            // Weights of every number above the cut's bin, relative to its bin's largest. Behind a cut
            // they are few: 2,048 logits at a time, those that count go to a queue and then to all
            // threads evenly. (64 rows of 32,000 of deviation 8 with top_k 1,000 and top_p 0.9: 78 us. When
            // this was done 334 became 91, the weights evaluated where they were loaded: every warp ran the long code for a lane or two, each at another place.)
            const uint32_t* x = static_cast<const uint32_t*>(p.logits) + (long long)row * p.vocab;
            const int i1 = (int)r.i1;
            auto load = [&](int i) { return i < i1 ? x[i] : 0x7fffffffu; };  // (NaN: none)
            // To units of 2^-43, rounded up where the rest exceeds a number that only the logit's index
            // gives (multiples of the golden ratio, modulo 1): equal logits, of which a row may have a
            // million, would all round alike to the nearest (5,000 distinct ones and 257,000 at e^-17 of
            // the largest in one bin: the sum off by 2^-23).
            auto add = [&](uint32_t key, uint32_t index) {
                const uint32_t anchor = min(key | 0xffffu, key_max);
                const F2 w = key == anchor ? F2{1.f, 0.f}
                                           : r.template relative<true>(
                                                 r.template capped<true>(K::value(key)),
                                                 r.template capped<true>(K::value(anchor)));
                const u64 fine = (u64)(__float2ll_rn(w.h * 0x1p62f) + __float2ll_rn(w.l * 0x1p62f));
                const u64 v = (fine + (index * 0x9e3779b9u >> 13)) >> 19;
                if (v) atomicAdd(mass + (key >> 16), v);
            };
            int i0 = (int)r.i0 + tid;
            uint32_t next[2] = {load(i0), load(i0 + kThreads)};
            if (cut_all) {
#pragma unroll 1
                for (; i0 < i1; i0 += kThreads) {
                    const uint32_t key = K::of(next[0]);
                    next[0] = next[1];
                    next[1] = load(i0 + 2 * kThreads);
                    if (key >= K::kLow && key <= K::kInf) add(key, (uint32_t)i0);
                }
            } else {
                uint32_t* queue = reinterpret_cast<uint32_t*>(s.before2 + kGather);  // [2 kThreads]
                lower_of = 0xffffffffu;  // (its sums were there)
                if (tid == 0) s.queued[0] = 0;
                __syncthreads();
#pragma unroll 1
                for (int b0 = (int)r.i0, turn = 0; b0 < i1; b0 += 2 * kThreads, turn ^= 1) {
                    const uint32_t now[2] = {next[0], next[1]};
                    i0 += 2 * kThreads;
                    next[0] = load(i0);
                    next[1] = load(i0 + kThreads);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t key = K::of(now[h]);
                        const bool counts = key <= K::kInf && key >> 16 > cut_bin;
                        const unsigned lanes = __ballot_sync(0xffffffffu, counts);
                        uint32_t at0 = 0;
                        if (lane == 0 && lanes) at0 = atomicAdd(&s.queued[turn], __popc(lanes));
                        at0 = __shfl_sync(0xffffffffu, at0, 0);
                        if (counts)
                            queue[at0 + __popc(lanes & ((1u << lane) - 1))] =
                                (uint32_t)(i0 + (h - 2) * kThreads);
                    }
                    __syncthreads();
                    const uint32_t n = s.queued[turn];
                    if (tid == 0) s.queued[turn ^ 1] = 0;
#pragma unroll 1
                    for (uint32_t k = tid; k < n; k += kThreads) add(K::of(x[queue[k]]), queue[k]);
                    __syncthreads();
                }
            }
            __threadfence();  // (the sums lie in global memory)
            cluster_barrier();
        }
        // kept weight of a bin
        auto bin_mass = [&](int g, int i) -> u64 {
            const uint32_t bin = (uint32_t)(g * 32 + i);
            if (bin > bin_max) return 0;
            if (F32) {
                if (!cut_all && bin <= cut_bin) return bin == cut_bin ? cut_mass : 0;
                if (!(s.live[g / 32] >> (g & 31) & 1u)) return 0;  // (never set to zero)
                const u64 v = *reinterpret_cast<volatile u64*>(mass + bin);
                if (!v) return 0;
                const F2 w = r.weight(min(bin << 16 | 0xffffu, key_max));
                // v <= 2^63 as a sum of three numbers of at most 24 bits
                const float a = (float)(v >> 40), b = (float)(v >> 20 & 0xfffffu),
                            c = (float)(v & 0xfffffu);
                return r.units(w * F2{a * 0x1p-3f, 0.f}, 1u) +
                       r.units(w * fast_sum(b * 0x1p-23f, c * 0x1p-43f), 1u);
            }
            const uint32_t n = kept_of(bin, r.bin_count(g, i));
            return n ? r.units(r.weight(bin), n) : 0;
        };
        for (int q = warp; rank + q * C < kGroups; q += kWarps) {
            const int g = rank + q * C;
            if (!(s.live[g / 32] >> (g & 31) & 1u)) continue;
            u64 m = bin_mass(g, lane);
            if (!__any_sync(0xffffffffu, m != 0)) continue;
            m = __shfl_sync(0xffffffffu, r.warp_sums(m), 31);
            if (lane < C) st_peer(peer_addr(&s.before[g], lane), m);
        }
        cluster_barrier();
        r.running_sums(s.before);
        const u64 all = s.before[kGroups - 1];

        // The place in the order where the running weight first is at least `need` (1..all); and
        // the running weight there. One warp looks into a group, the others wait for it.
        auto place = [&](u64 need, Cut& c, u64& sum) {
            const int d = r.reach(s.before, need);
            if (warp == 0) {
                const int g = kGroups - 1 - d;
                const u64 m = bin_mass(g, 31 - lane), x = r.warp_sums(m);
                const u64 base = d ? s.before[d - 1] : 0;
                const int l = __ffs(__ballot_sync(0xffffffffu, base + x >= need)) - 1;
                const uint32_t bin = (uint32_t)(g * 32 + 31 - l);
                if (lane == l) {
                    s.key = bin;
                    s.start = base + x - m;
                    s.m = m;
                    if (!F32) s.n = kept_of(bin, r.bin_count(g, 31 - l));
                }
            }
            __syncthreads();
            if (F32) {
                const uint32_t upper = s.key;
                const u64 start = s.start, m_bin = s.m;
                __syncthreads();
                if (gathers(upper)) {
                    const Entry e = gather(upper);
                    const u64 m = e.have && stays(e) ? r.units(r.weight(e.key), 1u) : 0;
                    const u64 run = r.sum_before(m) + m;
                    if (tid == kThreads - 1) s.m = run;
                    __syncthreads();
                    const u64 have = s.m;
                    const u64 rest = have ? min(max(m_bin ? need - start : 1, (u64)1), have) : 0;
                    if (have ? run - m < rest && rest <= run : tid == 0) {
                        s.key = e.key;
                        s.n = e.tie + 1;
                        s.index = e.index;
                        s.start = start + (have ? run : m_bin);
                    }
                    __syncthreads();
                    c = Cut{s.key, s.n};
                    sum = s.start;
                    drawn = s.index;
                    __syncthreads();
                    return;
                }
                drawn = 0xffffffffu;
                lower_masses(upper);
                // (the bin's weight was summed token by token, here value by value: the last units
                // may differ)
                const u64 have = s.before2[kGroups - 1];
                if (have == 0) {  // weights too small for a unit each: the bin's first token
                    uint32_t low, tie;
                    kth(1, low, tie);
                    c = Cut{upper << 16 | low, 1u};
                    sum = start + m_bin;
                    return;
                }
                const u64 rest = min(max(m_bin ? need - start : 1, (u64)1), have);
                const int d2 = r.reach(s.before2, rest);
                if (warp == 0) {
                    const int g2 = kGroups - 1 - d2;
                    const uint32_t key = upper << 16 | (uint32_t)(g2 * 32 + 31 - lane);
                    const uint32_t n = kept_of(key, r.bin_count(g2, 31 - lane));
                    const u64 m = n ? r.units(r.weight(key), n) : 0, x = r.warp_sums(m);
                    const u64 base = d2 ? s.before2[d2 - 1] : 0;
                    const int l = __ffs(__ballot_sync(0xffffffffu, base + x >= rest)) - 1;
                    if (lane == l) {
                        s.key = key;
                        s.start = start + base + x - m;
                        s.m = m;
                        s.n = n;
                        need = start + rest;
                    }
                    need = __shfl_sync(0xffffffffu, need, l);
                }
            }
            if (tid < 32) __syncwarp();
            if (tid == 0) {
                // the first tie i of n with start + (i + 1) m / n at least need
                const u64 m = s.m, n = s.n;
                const u64 gap = need > s.start ? need - s.start : 1;
                u64 i = 0;
                if (n > 1 && m) {  // (an estimate, off by one at most, and exact products)
                    const unsigned __int128 gn = (unsigned __int128)gap * n;
                    i = min((u64)((double)gap / (double)m * (double)n), n - 1);
                    while (i > 0 && (unsigned __int128)i * m >= gn) --i;
                    while (i < n - 1 && (unsigned __int128)(i + 1) * m < gn) ++i;
                }
                s.n = (uint32_t)(i + 1);
                // floor((i + 1) m / n), the quotient's and the remainder's parts apart
                s.start += i + 1 == n ? m : (i + 1) * (m / n) + (i + 1) * (m % n) / n;
            }
            __syncthreads();
            c.key = s.key;
            c.ties = s.n;
            sum = s.start;
            __syncthreads();
        };

        Cut end = cut;  // what is kept in the end, and its weight
        bool end_all = cut_all;
        u64 kept = all;
        // the cut by top_p with min_p's behind it, and then the draw (one copy of the search)
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
            u64 need = 0;
            if (turn == 1) {
                need = min((u64)((double)u * (double)kept) + 1, kept);  // the weight passes u kept
            } else if (top_p <= 0.f) {
                end = Cut{key_max, 1u};
                end_all = false;
                kept = r.units(F2{1.f, 0.f}, 1u);
            } else if (top_p < 1.f) {
                need = min(max((u64)ceil((double)top_p * (double)all), (u64)1), all);
            }
            Cut c{0u, 0u};
            u64 sum = 0;
            if (need) place(need, c, sum);
            if (turn == 1) {
                draw_key = c.key;
                draw_tie = c.ties - 1;
                break;
            }
            if (need) {
                end = c;
                end_all = false;
                kept = sum;
            }
            if (min_p > 0.f) {
                // the smallest key whose weight is at least min_p (the largest candidate's at any rate)
                if (warp == 0) {
                    uint32_t lo = K::kLow, hi = key_max;
                    while (lo < hi) {
                        const uint32_t step = max((hi - lo) / 32u, 1u);
                        const uint32_t off = (uint32_t)(lane + 1) * step;
                        bool ok = off <= hi - lo;
                        if (ok) {
                            const F2 w = r.weight(hi - off);
                            ok = w.h > min_p || (w.h == min_p && w.l >= 0.f);
                        }
                        const unsigned bad = ~__ballot_sync(0xffffffffu, ok);
                        const uint32_t n = bad ? (uint32_t)__ffs(bad) - 1 : 32u;
                        const uint32_t past = (n + 1) * step;  // not ok there, or out of range
                        if (n < 32 && past <= hi - lo) lo = hi - past + 1;
                        hi -= n * step;
                        if (step == 1 && n < 32) break;
                    }
                    if (lane == 0) s.key = hi;
                }
                __syncthreads();
                const uint32_t floor_key = s.key;
                __syncthreads();
                if (end_all || floor_key > end.key) {
                    // everything from the floor up (its own tokens too, if there are any)
                    const uint32_t bin = F32 ? floor_key >> 16 : floor_key;
                    u64 from = 0;  // fp32: weight of the bin's numbers from the floor up
                    const bool few = gathers(bin);
                    if (few) {
                        const Entry e = gather(bin);
                        const u64 m = e.have && e.key >= floor_key && stays(e)
                                          ? r.units(r.weight(e.key), 1u) : 0;
                        const u64 run = r.sum_before(m) + m;
                        if (tid == kThreads - 1) s.m = run;
                        __syncthreads();
                        from = s.m;
                        __syncthreads();
                    } else if (F32) {
                        lower_masses(bin);
                    }
                    if (warp == 0) {
                        const int g = (int)(bin / 32), d = kGroups - 1 - g;
                        const bool above = (uint32_t)(g * 32 + lane) > bin ||
                                           (!F32 && (uint32_t)(g * 32 + lane) == bin);
                        u64 m = r.warp_sums(above ? bin_mass(g, lane) : (u64)0);
                        m = __shfl_sync(0xffffffffu, m, 31) + (d ? s.before[d - 1] : 0);
                        if (few) {
                            m += from;
                        } else if (F32) {
                            const uint32_t low = floor_key & 0xffffu;
                            const int g2 = (int)(low / 32), d2 = kGroups - 1 - g2;
                            const uint32_t key = bin << 16 | (uint32_t)(g2 * 32 + lane);
                            const uint32_t c = key >= floor_key ? r.bin_count(g2, lane) : 0u;
                            const u64 x = r.warp_sums(c ? r.units(r.weight(key), c) : (u64)0);
                            m += __shfl_sync(0xffffffffu, x, 31) + (d2 ? s.before2[d2 - 1] : 0);
                        }
                        if (lane == 0) s.m = m;
                    }
                    __syncthreads();
                    kept = min(s.m, all);
                    __syncthreads();
                    end_all = false;
                }
            }
        }
    }
    if (drawn != 0xffffffffu) {
        if (rank == 0 && tid == 0) p.token[row] = (int32_t)drawn;
        return;
    }
    if (F32) refine(draw_key >> 16);

    // Which CTA's slice holds occurrence draw_tie of draw_key: every CTA reads the slices' counts.
    const uint32_t bin = F32 ? draw_key & 0xffffu : draw_key;
    uint32_t mine = 0, before = 0;
    for (int q = 0; q < C; ++q) {
        const uint32_t c = ld_peer(peer_addr(hist + (bin >> 1), q)) >> (16 * (bin & 1)) & 0xffffu;
        if (q < rank) before += c;
        if (q == rank) mine = c;
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
    if (draw_tie < before || draw_tie >= before + mine) return;
    // That occurrence within the slice: every thread counts it in a run of 16-byte pieces, and the
    // one whose run holds it looks again.
    constexpr int E = F32 ? 4 : 8;
    const long long b0 = (long long)row * p.vocab + r.i0, b1 = (long long)row * p.vocab + r.i1;
    const long long end = (long long)p.batch * p.vocab;
    auto hits_of = [&](long long v) {  // of piece v, as a bit per element
        const long long at = v * E;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (at + E <= end) {
            const uint4 x = reinterpret_cast<const uint4*>(p.logits)[v];
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
        } else {  // the last elements of the array
            for (int e = 0; e < E && at + e < end; ++e) {
                if (F32) w[e] = static_cast<const uint32_t*>(p.logits)[at + e];
                else w[e / 2] |= (uint32_t) static_cast<const uint16_t*>(p.logits)[at + e] << 16 * (e & 1);
            }
        }
        uint32_t hits = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t bits = F32 ? w[e & 3] : w[e / 2] >> 16 * (e & 1) & 0xffffu;
            if (K::of(bits) == draw_key && at + e >= b0 && at + e < b1) hits |= 1u << e;
        }
        return hits;
    };
    const long long first = b0 / E, last = (b1 + E - 1) / E;
    const long long run = (last - first + kThreads - 1) / kThreads;
    const long long v0 = min(first + tid * run, last), v1 = min(v0 + run, last);
    uint32_t count = 0;
#pragma unroll 4
    for (long long v = v0; v < v1; ++v) count += __popc(hits_of(v));
    const uint32_t ex = r.sum_before(count), left = draw_tie - before;
    if (left < ex || left >= ex + count) return;
    uint32_t skip = left - ex;
    for (long long v = v0; v < v1; ++v) {
        uint32_t hits = hits_of(v);
        const uint32_t c = __popc(hits);
        if (skip < c) {
            for (; skip > 0; --skip) hits &= hits - 1;
            p.token[row] = (int32_t)(v * E + __ffs(hits) - 1 - (long long)row * p.vocab);
            return;
        }
        skip -= c;
    }
}

// Every cluster draws rows i, i + clusters, ... of those that are its launch's: all (kAlone), those
// that the list launch left to it (kAfterList), or first those that the lists do not take on, without
// waiting for them, and then those that they left open (kAhead: the list launch itself started with
// everything before it complete, and its CTAs leave one by one; the first rows are drawn on the SMs
// that they have left. 64 mixed rows of 262,144 68.4 -> 61.1 us, but one row with a list 13.9 ->
// 14.2 and nine fp32 rows 32.3 -> 33.7). The i-th such row is found from the rows' filters and flags,
// which nobody changes here.
enum { kAlone, kAfterList, kAhead };
template <bool F32>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleParams p, int C,
                                                             int order) {
    pdl_launch_dependents();
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& s = *reinterpret_cast<Shared*>(smem);
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem + (sizeof(Shared) + 15) / 16 * 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool lists = false;  // the lists took row b on
#pragma unroll 1
    for (int pass = order == kAhead ? 0 : 1; pass < 2; ++pass) {
        if (pass == 1) pdl_wait();
        int passed = 0;  // such rows before row b0
        int i = blockIdx.x / C;
        for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
            const int b = b0 + tid;
            bool is = b < p.batch;
            if (is && order == kAhead) {
                if (pass == 0 || p.batch > kThreads) {  // (else as in the first pass)
                    Filters f;
                    lists = !f.load(p, b) || f.listed<F32>(p.softcap);
                }
                is = pass == 0 ? !lists : lists && p.open[b];
            } else if (is && order == kAfterList) {
                is = p.open[b];
            }
            const unsigned word = __ballot_sync(0xffffffffu, is);
            if (lane == 0) s.open[warp] = word;
            __syncthreads();
            int base = 0, all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) base += __popc(s.open[w]);
                all += __popc(s.open[w]);
            }
            for (; i < passed + all; i += gridDim.x / C) {
                if (is && passed + base + __popc(word & ((1u << lane) - 1)) == i) s.row = b;
                __syncthreads();
                const int row = s.row;
                draw_row<F32>(p, s, hist, C, row);
                cluster_barrier();  // (shared memory is used anew)
            }
            passed += all;
            __syncthreads();
        }
    }
}

// Launches of `clusters` clusters of C CTAs.
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Launch(int clusters, int C, int threads, size_t smem, bool early, cudaStream_t st) {
        cfg.gridDim = dim3((unsigned)clusters * C);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)C;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = early ? 2 : 1;
    }
};

// What is asked or set once per device (the same values every time).
struct DeviceState {
    std::atomic<bool> configured{false};
    std::atomic<int> at_once[kMaxCtas + 1] = {};  // clusters of C CTAs that the GPU holds, or 0
};
constexpr int kDevices = 64;

template <class Kernel>
cudaError_t configure(Kernel* kernel, DeviceState& d, int max_smem) {
    if (d.configured.load(std::memory_order_relaxed)) return cudaSuccess;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) d.configured.store(true, std::memory_order_relaxed);
    return e;
}

static_assert((sizeof(Shared) + 15) / 16 * 16 + kBins * 2 + (kGroups + 4) / 5 * 128 <= 227 * 1024,
              "a cluster of five fits");
size_t row_smem(int C) {
    return (sizeof(Shared) + 15) / 16 * 16 + kBins * 2 +
           (C > 1 ? (size_t)(kGroups + C - 1) / C * 32 * 4 : 0);
}

// In us, bf16, 1 / 5 / 8 / 11 / 16 CTAs per row: one row of 262,144 - / 32.5 / 29.7 / 26.8 / 27.8, of
// 32,000 41.5 / 25.1 / 24.1 / 24.4 / 25.6; 16 rows - / 40.5 / 56.9 / 55.8 / 79.6 and 45.5 / 25.3 /
// 45.7 / 46.6 / 71.3; 64 rows - / 112 / 146 / 218 / 260 (6: 103) and 45.7 / 71.0 / 111.8 / 179.9 /
// 231.9.
// CTAs per row: one, or 5 to 16 (so that the merged counts fit beside the histogram), no slice above
// what a 16-bit counter holds; as many as take the batch the least time, in rounds of the clusters
// that the GPU holds at once.
template <bool F32>
cudaError_t row_ctas(const SampleParams& p, DeviceState& d, int* ctas, int* clusters) {
    double best = 0.0;
    *ctas = 0;
    for (int c = 1; c <= kMaxCtas; c = c == 1 ? 5 : c + 1) {
        const int slice = (p.vocab + c - 1) / c;
        if (slice > 65535) continue;
        int fit = d.at_once[c].load(std::memory_order_relaxed);
        if (fit == 0) {
            Launch l(1, c, kThreads, row_smem(c), true, nullptr);
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&fit, sample_kernel<F32>, &l.cfg);
            if (e != cudaSuccess) return e;
            if (fit < 1) fit = -1;
            d.at_once[c].store(fit, std::memory_order_relaxed);
        }
        if (fit < 1) continue;
        const double rounds = (p.batch + fit - 1) / fit;
        const double cost = rounds * ((c == 1 ? kAloneCost : kClusterCost) + slice);
        if (*ctas == 0 || cost < best) {
            best = cost;
            *ctas = c;
            *clusters = p.batch < fit ? p.batch : fit;
        }
    }
    return *ctas ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <bool F32>
cudaError_t launch(const SampleParams& p, cudaStream_t st) {
    static DeviceState lists[kDevices], rows[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return cudaErrorInvalidDevice;
    // the list can decide rows only if some may have a short top_k (or are fp32 without a cap)
    const bool listed = p.top_k != nullptr || (F32 && !(p.softcap > 0.f));
    if (listed) {
        // CTAs per row, in us with 1 / 2 / 4 / 8 / 16: bf16 with top_k 200, 262,144 logits: one row
        // - / 31.2 / 22.3 / 18.2 / 19.0, 64 - / 37.3 / 28.5 / 27.0 / 41.7 (clusters of 16 find few
        // places), 400 - / 92.7 / 87.3 / 96.7 / 172; 32,000 logits: 64 rows 26.8 / 20.8 / 20.7 /
        // 21.8 / 36.2, 400 39.4 / 41.9 / 47.3 / 62.9 / 139. fp32, top_k 20, 262,144 logits: one row
        // - / 42.0 / 27.8 / 20.4 / 17.8.
        const int slice = p.batch > 100 ? 65536 : 8192, most = F32 && p.batch <= 8 ? kMaxCtas : 8;
        const int c = (p.vocab + slice - 1) / slice, C = c > most ? most : c;
        cudaError_t e = configure(list_kernel<F32>, lists[dev], 64 * 1024);
        if (e != cudaSuccess) return e;
        // Not ahead of the launch before it. sample_kernel's first pass (kAhead) relies on that: it reads
        // logits and filters and writes tokens and sums before it waits for the lists, so everything
        // before these has to be complete when they start. It is faster too: the CTAs of the launch
        // before may fill most SMs, and the lists would crowd on the others (22.8 us for 8 rows of
        // 262,144 logits against 16.1).
        Launch l(p.batch, C, kListThreads, sizeof(ListShared), false, st);
        e = cudaLaunchKernelEx(&l.cfg, list_kernel<F32>, p, C);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = configure(sample_kernel<F32>, rows[dev], 227 * 1024);
    if (e != cudaSuccess) return e;
    int C = 0, clusters = 0;
    e = row_ctas<F32>(p, rows[dev], &C, &clusters);
    if (e != cudaSuccess) return e;
    Launch l(clusters, C, kThreads, row_smem(C), true, st);
    const int order = !listed ? kAlone : p.batch < 16 ? kAfterList : kAhead;
    return cudaLaunchKernelEx(&l.cfg, sample_kernel<F32>, p, C, order);
}

}  // namespace

size_t sample_workspace(int batch, int fp32) {
    return ((size_t)batch * 4 + 15) / 16 * 16 + (fp32 ? (size_t)batch * kBins * 8 : 0);
}

cudaError_t launch_sample(const SampleParams& p, int fp32, cudaStream_t st) {
    return fp32 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace gemma
