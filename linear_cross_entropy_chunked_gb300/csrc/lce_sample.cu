// Drawing one token per row of logits Z [N, ld] (bf16, fp16 or fp32) by inversion
// from one given uniform number u in [0, 1) per row.
//
// With m the row's largest logit, x_i = (m - z_i) / temperature and w_i = exp(-x_i):
//   * order the tokens by logit, largest first, equal logits by index;
//   * top-k keeps the first k; top-p keeps, of those, each token before which less
//     than p of their weight lies; min-p keeps w_i >= min_p. Each keeps a prefix of
//     the order and never less than its first token;
//   * the token is the lowest index i (in index order) at which the kept weight up
//     to and including i exceeds u times all kept weight; its log-probability is
//     -x_i - log(sum of kept w).
//
// Arithmetic. A token is a whole number: it must not depend on the order of a
// sum, and a border of the cumulative distribution must lie where the formula
// puts it. So weights are whole numbers, w_i in units of 2^-43 (64-bit sums
// of up to 2^20 tokens are exact and the same in any order), and exp is computed
// to a relative error of about 2^-31. A weight is rounded to its unit, to nearest, so that the errors of a
// row's tokens have no common sign. The chance that u falls on the wrong side of a border, which is the sum
// over all borders of how far they are off: 1e-8 for 2^17 equally likely tokens, 1e-6 for 128256 normal
// logits with a few likely ones at temperature 0.7, 5e-7 for 128256 tokens 16 below a single likely one, 2e-5
// for 2^20 of those. (Weights cut to their unit would have it at 8e-5, 5e-4 and 2e-2 in the last three, the
// exponential in fp32 with exact sums at 4e-4, 4e-6 and 2e-4, an fp32 softmax at about 1e-2. Equal
// logits are rounded alike: 1e-4 and 7e-3 for 128256 and 2^20 of them 16 below a single one.)
//
// Bound: one read of the logits. A cluster of CTAs holds a row in shared memory,
// so every later pass (the search for the cut, the sums, the draw) stays on chip; the
// CTAs exchange maxima, histograms and sums through distributed shared memory. Rows
// longer than the cluster's shared memory, and long rows of large batches, for which small
// clusters are faster, are read again from L2 instead.
// Measured: 1 x 32000 bf16 5.8 us, 64 x 128256 bf16 20 us, 256 x 128256 bf16 65 us and fp32 70 us
// (1.9 TB/s; the read alone would take 19 us). What takes the time: about 36 instructions per logit,
// nearly all for the exponential (3 of them round it; with cut weights the last two take 62 and 67 us), and a
// CTA's start, exchanges and tail, which the second CTA of an SM
// covers in part. 64 x 128256 bf16 with top-k 50 takes 17 us; with top-p 0.9 of flat rows, whose
// cut lies beyond the list, 63 us, in three parts: the histogram, the keys of its bin, and the
// sums of what is kept with the draw. (Figures further down that compare variants of this kernel were taken
// with cut weights.)
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "lce_internal.h"
#include "lce_ptx.cuh"

namespace lce {

constexpr int SMP_THREADS = 512;
constexpr int SMP_WARPS = SMP_THREADS / 32;
constexpr int SMP_MAX_CLUSTER = 8;
constexpr int SMP_BINS = 256;
constexpr int SMP_ONE_SHIFT = 43;                    // weight of the largest logit: 2^43
constexpr float SMP_X_END = 31.f;                    // exp(-31) < 2^-44 rounds to weight 0
// Bins of x in which a cut is searched: half of them up to 8, half from there to 31.
constexpr float SMP_X_MID = 8.f;
// Parts of a row whose largest logits are exchanged.
constexpr int SMP_PARTS = SMP_MAX_CLUSTER * SMP_WARPS;
// A short list of the largest logits, in which most cuts lie: per CTA, and in all.
constexpr int SMP_LIST_CTA = 256, SMP_LIST = SMP_THREADS;
constexpr int SMP_BIN_CTA = 2048;                    // logits of a searched bin that a CTA keeps apart
constexpr int SMP_MAX_CTA = 1 << 17;                 // logits of a CTA: its histograms' limbs fit 32 bits
constexpr int SMP_SWEEPS = SMP_MAX_CTA / SMP_WARPS / 256;
static_assert(SMP_SWEEPS == 32, "one lane per sweep of a warp");
constexpr int SMP_LIMB = 15;                         // bits per limb of a weight: 2^17 limbs fit 32 bits

constexpr int SMP_STEP_BITS = 8, SMP_STEPS = 1 << SMP_STEP_BITS;   // the exponential's table: 2^(-j / 256)

constexpr float SMP_ROUND = 12582912.f;              // 1.5 * 2^23

// Constants of the exponential, from their definitions on the host. Pairs: packed
// arithmetic takes them from the parameters as they are.
SampleTables make_sample_tables() {
    SampleTables t;
    const double ln2 = std::log(2.0);
    for (int j = 0; j < SMP_STEPS; ++j)
        t.fix[j] = static_cast<unsigned>(std::nearbyint(std::ldexp(std::exp2(-j / static_cast<double>(SMP_STEPS)), 31)));
    // ln(2) / 256 in three parts: 10 bits (its product with a whole number below
    // 2^14 is exact), 24 bits, and the rest
    const double step = ln2 / SMP_STEPS;
    int e;
    std::frexp(step, &e);
    const double ulp = std::ldexp(1.0, e - 10);
    const double c1 = std::floor(step / ulp) * ulp;
    const float c2 = static_cast<float>(step - c1);
    auto two = [](double v) { return make_float2(static_cast<float>(v), static_cast<float>(v)); };
    t.c1 = two(c1);
    t.c2 = two(c2);
    t.mc3 = two(-(step - c1 - static_cast<double>(c2)));
    t.ninv = two(-SMP_STEPS / ln2);
    // 1.5 * 2^23 rounds what it is added to to a whole number n, kept in its low bits; 19 is
    // added to the n / 256 there: the shift from units of 2^-62 to 2^-43
    const float magic = SMP_ROUND + 19 * SMP_STEPS;
    t.magic = two(magic);
    t.mmagic = two(-magic);
    // exp(r) - 1 = r (1 + r (1 / 2 + r / 6)) in units of 2^-31, to 2^-42
    const double S = 2147483648.0;
    t.p3 = two(S / 6);
    t.p2 = two(S / 2);
    t.p1 = two(S);
    t.round = two(SMP_ROUND);
    return t;
}

namespace {

typedef unsigned long long u64;

// ------------------------------------------------------------------ logits in vectors of 8

__device__ __forceinline__ void smp_unpack(const uint4 &u, float (&x)[8], const __nv_bfloat16 *) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        x[2 * q] = __uint_as_float(w[q] << 16);
        x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
}
__device__ __forceinline__ void smp_unpack(const uint4 &u, float (&x)[8], const __half *) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
        x[2 * q] = f.x;
        x[2 * q + 1] = f.y;
    }
}
// 8 logits at p (aligned to 16 bytes), as they are.
template <typename T> __device__ __forceinline__ void smp_load_vec(const T *p, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        smp_unpack(*reinterpret_cast<const uint4 *>(p), x, static_cast<const T *>(nullptr));
    }
}
// 8 logits of 16 bits from any address, by words where they are aligned and no byte beside them: of an odd
// address the first and the last logit come alone.
__device__ __forceinline__ uint4 smp_load_words(const void *p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a & 2u) {
        const uint32_t first = *static_cast<const uint16_t *>(p), last = static_cast<const uint16_t *>(p)[7];
        const uint32_t *u = reinterpret_cast<const uint32_t *>(a + 2);
        const uint32_t w0 = u[0], w1 = u[1], w2 = u[2];
        return make_uint4(first | (w0 << 16), __funnelshift_r(w0, w1, 16), __funnelshift_r(w1, w2, 16),
                          (w2 >> 16) | (last << 16));
    }
    const uint32_t *u = reinterpret_cast<const uint32_t *>(a);
    return make_uint4(u[0], u[1], u[2], u[3]);
}
// 8 logits from global memory; those past `n` are -infinity. (Rows that start anywhere by words:
// 512 x 50257 fp16 65.6 us; with cut weights 63, and value by value 67.9.)
template <typename T>
__device__ __forceinline__ void smp_load_global(const T *p, int n, bool aligned, float (&x)[8]) {
    if (aligned && n >= 8) {
        smp_load_vec<T>(p, x);
    } else if (sizeof(T) == 2 && n >= 8) {
        if constexpr (sizeof(T) == 2) smp_unpack(smp_load_words(p), x, p);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < n ? static_cast<float>(p[j]) : -INFINITY;
    }
}

// The same as they are, to be copied (16-bit types packed), and the largest, NaN aside.
template <typename T> struct SmpRaw {
    uint32_t u[4];
    __device__ __forceinline__ void load(const T *p, int n, bool aligned) {
        if (aligned && n >= 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
        } else if (n >= 8) {
            const uint4 v = smp_load_words(p);
            u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
        } else {
            constexpr uint32_t MINUS_INF = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                u[j] = (2 * j < n ? h[2 * j] : MINUS_INF) | ((2 * j + 1 < n ? h[2 * j + 1] : MINUS_INF) << 16);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ float largest() const {
        using V = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
        const V *v = reinterpret_cast<const V *>(u);
        const V m = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
        return fmaxf(static_cast<float>(m.x), static_cast<float>(m.y));
    }
};
template <> struct SmpRaw<float> {
    float x[8];
    __device__ __forceinline__ void load(const float *p, int n, bool aligned) { smp_load_global<float>(p, n, aligned, x); }
    __device__ __forceinline__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ __forceinline__ float largest() const {
        float m = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, x[j]);
        return m;
    }
};

// Order-preserving whole number of a logit. 16-bit types: the 32-bit pattern's low
// bits, which are the same for all values of the type and sign, are dropped.
template <typename T> struct SmpKey;
template <> struct SmpKey<__nv_bfloat16> { static constexpr int DROP = 16; };
template <> struct SmpKey<__half> { static constexpr int DROP = 13; };
template <> struct SmpKey<float> { static constexpr int DROP = 0; };

template <typename T> __device__ __forceinline__ uint32_t smp_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);   // (-0 is equal to +0)
    return (b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) >> SmpKey<T>::DROP;
}
template <typename T> __device__ __forceinline__ float smp_unkey(uint32_t key) {
    constexpr int DROP = SmpKey<T>::DROP;
    uint32_t b = key << DROP;
    if (b >> 31) return __uint_as_float(b ^ 0x80000000u);
    return __uint_as_float((~b) & ~((1u << DROP) - 1u));
}

// ------------------------------------------------------------------ weights

constexpr u64 SMP_ONE = 1ull << SMP_ONE_SHIFT;

struct SmpRow {
    float m, ih, il;       // largest logit; 1 / temperature in two parts
};

// x = (m - z) / temperature, rounded: the same monotone function wherever it is used.
__device__ __forceinline__ float smp_x(float z, const SmpRow &r) {
    return (r.m - z) * r.ih;
}

// exp(-(m - z) / temperature) in units of 2^-43 of two logits (in packed fp32 arithmetic, which
// halves the instructions). x is carried in two floats (-nx + xl, from m - z = d + dl exactly);
// x = n ln(2) / 256 - rr, exp(-x) = 2^-(n / 256) * (1 + q) with q = exp(rr) - 1, |rr| < 0.0014. (With -x in
// place of x no product by -1 is needed for xl: 256 x 128256 fp32 69.9 us for 72.5.)
// Table and 1 + q are whole numbers of 31 bits (2^-31), their product exact; half a unit is
// added to it, and the shift by n / 256 leaves whole units. The largest logit's weight is 2^43 exactly. (A table
// of 64 needs one more term of q, and a conversion for the whole number of 1 + q that here
// comes out of the last addition's rounding: |q| < 2^22 units.) NaN has weight 0.
__device__ __forceinline__ u64 smp_finish(float kf, float q31, const unsigned *tab) {
    const unsigned n = static_cast<unsigned>(__float_as_int(kf));
    const unsigned f = static_cast<unsigned>(__float_as_int(q31)) + (0x80000000u - 0x4b400000u);
    // 19 and more. From 64 on, and for any x beyond, infinite ones and NaN too, PTX's shift gives 0
    // whatever is shifted (64 x 128256 bf16 20.3 us; with x held at 32 first 20.6)
    const unsigned shift = (n - 0x4b400000u) >> SMP_STEP_BITS;
    u64 half, w;
    asm("shl.b64 %0, %1, %2;" : "=l"(half) : "l"(1ull), "r"(shift - 1));
    asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(static_cast<u64>(tab[n & (SMP_STEPS - 1)]) * f + half), "r"(shift));
    return w;
}
__device__ __forceinline__ void smp_weight2(float z0, float z1, const SmpRow &r, const SampleTables &c,
                                            const unsigned *tab, u64 &w0, u64 &w1) {
    auto two = [](float v) { return make_float2(v, v); };
    const float2 z = make_float2(z0, z1), m = two(r.m), minus = two(-1.f), ih = two(r.ih);
    const float2 d = __ffma2_rn(z, minus, m);
    const float2 bb = __ffma2_rn(m, minus, d);
    const float2 dl = __ffma2_rn(__fadd2_rn(z, bb), minus, __ffma2_rn(__ffma2_rn(bb, minus, d), minus, m));
    const float2 nx = __fmul2_rn(d, two(-r.ih));
    float2 xl = __ffma2_rn(d, ih, nx);
    xl = __ffma2_rn(d, two(r.il), xl);
    xl = __ffma2_rn(dl, ih, xl);
    const float2 k = __ffma2_rn(nx, c.ninv, c.magic);
    const float2 nf = __fadd2_rn(k, c.mmagic);
    xl = __ffma2_rn(nf, c.mc3, xl);
    float2 rr = __ffma2_rn(nf, c.c1, nx);               // (exact wherever the weight is not 0)
    rr = __ffma2_rn(xl, minus, __ffma2_rn(nf, c.c2, rr));
    float2 q = __ffma2_rn(rr, c.p3, c.p2);
    q = __ffma2_rn(rr, q, c.p1);
    q = __ffma2_rn(rr, q, c.round);
    w0 = smp_finish(k.x, q.x, tab);
    w1 = smp_finish(k.y, q.y, tab);
}
__device__ __forceinline__ u64 smp_weight(float z, const SmpRow &r, const SampleTables &c, const unsigned *tab) {
    u64 a, b;
    smp_weight2(z, z, r, c, tab, a, b);
    return a;
}

// floor(f * s) and ceil(f * s) for 0 <= f < 1, exactly.
__device__ __forceinline__ u64 smp_mul_floor(float f, u64 s, bool ceil) {
    const uint32_t b = __float_as_uint(f);
    const int ex = static_cast<int>(b >> 23);           // f >= 0
    const u64 man = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int sh = 150 - (ex ? ex : 1);                 // f = man * 2^-sh, sh >= 24
    const u64 lo = man * s, hi = __umul64hi(man, s);    // < 2^88
    u64 q;
    bool rest;
    if (sh >= 128) {
        q = 0;
        rest = (lo | hi) != 0;
    } else if (sh >= 64) {
        const int k = sh - 64;
        q = hi >> k;
        rest = lo != 0 || (k && (hi << (64 - k)) != 0);
    } else {
        q = (lo >> sh) | (hi << (64 - sh));
        rest = (lo << (64 - sh)) != 0;
    }
    return q + (ceil && rest ? 1ull : 0ull);
}

// ------------------------------------------------------------------ cluster exchange

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                              uint32_t d) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t smp_cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ u64 shfl_up64(u64 v, int o) {
    return __shfl_up_sync(0xffffffffu, v, o);
}
__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What one CTA knows of its part of the row.
struct alignas(16) SmpSums {
    u64 w;                 // weight of all
    u64 wlist;             // ... of the logits on the list
    uint32_t list;         // logits on the list (more than SMP_LIST_CTA: it overflowed)
};
struct SmpShared {
    uint32_t hist[2][4][SMP_BINS];        // counts, three limbs of the weights; read by the peers
    float wmax[SMP_PARTS];                // largest logits of the warps' parts, of all warps of the cluster
    SmpSums sums[SMP_MAX_CLUSTER];        // of every CTA of the cluster
    uint4 wslot[SMP_MAX_CLUSTER * SMP_WARPS];   // per warp of the cluster: sum above the cut, ties
    union {
        struct {
            u64 list[SMP_LIST_CTA];            // key and inverted index; rank 0 reads the peers'
            u64 all[SMP_LIST], allw[SMP_LIST]; // rank 0: the whole list, and its weights
        };
        struct {                               // logits in the bin that is searched: key, warp
            uint32_t bin_key[SMP_BIN_CTA];
            uint8_t bin_warp[SMP_BIN_CTA];
        };
    };
    u64 bin_w[SMP_WARPS];                 // of each warp, from those: kept weight above the cut, ties
    uint32_t bin_t[SMP_WARPS];
    u64 l0w[SMP_BINS], rw[SMP_BINS];      // weight before each bin: first level, refinement
    uint32_t l0c[SMP_BINS], rc[SMP_BINS]; // count before each bin
    u64 wsum[SMP_WARPS];
    uint32_t csum[SMP_WARPS];
    u64 bw;                               // the bin found: weight and count before it
    uint32_t bc;
    int bin;
    SmpSums part[SMP_WARPS];              // of every warp of this CTA
    uint32_t listed;                      // entries of `list` (or more, if it overflowed)
    float t0;
    u64 sweep_w[SMP_SWEEPS];              // sums of the sweeps over one warp's part
    uint32_t sweep_t[SMP_SWEEPS];
    unsigned tab[SMP_STEPS];
};

// The warp's part of the row: `n` logits from index `first` on, in shared memory
// (filled up to a multiple of 8 with -infinity) or in global memory.
template <typename T, bool SMEM> struct SmpChunk {
    const T *p;
    int n;
    bool aligned;
    // The largest logits share the row (one is +infinity, or 1 / temperature is not finite): they
    // are seen as 0, all others as -infinity.
    bool only_max;
    float m;
    __device__ __forceinline__ void load(int i, float (&x)[8]) const {
        load_plain(i, x);
        if (only_max) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] == m ? 0.f : -INFINITY;
        }
    }
    __device__ __forceinline__ void load_plain(int i, float (&x)[8]) const {
        if constexpr (SMEM) {
            if (i < n) {
                smp_load_vec<T>(p + i, x);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = -INFINITY;
            }
        } else {
            smp_load_global<T>(p + i, n - i, aligned, x);
        }
    }
};

// Adds a logit's weight and count to bin b of the histogram.
__device__ __forceinline__ void smp_hist_add(uint32_t (*hist)[SMP_BINS], int b, bool counts, bool weights, u64 w) {
    constexpr uint32_t M = (1u << SMP_LIMB) - 1u;
    if (counts) atomicAdd(&hist[0][b], 1u);
    if (weights) {
        atomicAdd(&hist[1][b], static_cast<uint32_t>(w) & M);
        atomicAdd(&hist[2][b], static_cast<uint32_t>(w >> SMP_LIMB) & M);
        const uint32_t top = static_cast<uint32_t>(w >> (2 * SMP_LIMB));
        if (top) atomicAdd(&hist[3][b], top);
    }
}

// SEARCH: some row has a top-k or a top-p. (Without the search's code a plain draw needs fewer
// registers: 256 x 128256 bf16 60.3 us, with it 67.0; 1 x 32000 5.6 and 7.3.)
template <typename T, bool SMEM, bool SEARCH>
__global__ void __launch_bounds__(SMP_THREADS, 2)
    lce_sample_kernel(const SampleParams p, const __grid_constant__ SampleTables tabs, const int chunk) {
    extern __shared__ __align__(128) uint8_t smp_dyn[];
    __shared__ SmpShared sh;
    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    const uint32_t rank = cluster_ctarank(), cl = smp_cluster_size();
    const long long r = blockIdx.x / cl;

    // settings of the row
    float temperature = p.temperature ? p.temperature[r] : p.temperature_all;
    const int top_k = p.top_k ? p.top_k[r] : p.top_k_all;
    const float top_p = p.top_p ? p.top_p[r] : p.top_p_all;
    const float min_p = p.min_p ? p.min_p[r] : p.min_p_all;
    const bool greedy = !(temperature > 0.f);
    const float u = p.u[r];

    cluster_arrive();   // waited for before the first write to a peer: it has started
    if (t < SMP_STEPS) sh.tab[t] = tabs.fix[t];

    // the warp's logits: into shared memory, and the largest (a NaN is never it, nor above any bound)
    const long long first = (static_cast<long long>(rank) * SMP_WARPS + w) * chunk;
    const long long left = p.V - first;
    const int n = left <= 0 ? 0 : left < chunk ? static_cast<int>(left) : chunk;
    const T *row = static_cast<const T *>(p.Z) + r * p.ld + (n > 0 ? first : 0);
    const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    SmpChunk<T, SMEM> ck;
    ck.n = n;
    ck.aligned = aligned;
    ck.only_max = false;
    ck.m = 0.f;
    float m = -INFINITY;
    if constexpr (SMEM) {
        T *mine = reinterpret_cast<T *>(smp_dyn) + static_cast<size_t>(w) * chunk;
        for (int i0 = l * 8; i0 < n; i0 += 4 * 256) {
            SmpRaw<T> x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i0 + q * 256 < n) x[q].load(row + i0 + q * 256, n - i0 - q * 256, aligned);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i0 + q * 256 < n) {
                    x[q].store(mine + i0 + q * 256);
                    m = fmaxf(m, x[q].largest());
                }
        }
        ck.p = mine;
    } else {
        ck.p = row;
        for (int i0 = l * 8; i0 < n; i0 += 4 * 256) {   // (loads of four sweeps under way at once)
            SmpRaw<T> x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)   // (-infinity past the end)
                x[q].load(row + i0 + q * 256, n - i0 - q * 256, aligned);
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, x[q].largest());
        }
    }
    const int steps = (n + 255) / 256;   // sweeps of the warp over its logits

    // Every warp gives its largest logits, of `sub` parts of it, to every CTA: SMP_PARTS in all,
    // whatever the cluster's size
    const int sub = SMP_MAX_CLUSTER / static_cast<int>(cl), group = 4 * static_cast<int>(cl);   // parts, lanes of one
    for (int o = 1; o < group; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int entries = static_cast<int>(cl) * SMP_WARPS, me = static_cast<int>(rank) * SMP_WARPS + w;
    cluster_wait();
    if (l % group < static_cast<int>(cl)) st_cluster_f32(map_to_rank(&sh.wmax[me * sub + l / group], l % group), m);
    cluster_sync_all();
    constexpr int PER_LANE = SMP_PARTS / 32;
    float wm[PER_LANE];   // parts 4 l .. 4 l + 3
    m = -INFINITY;
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        wm[q] = sh.wmax[l * PER_LANE + q];
        m = fmaxf(m, wm[q]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));

    if (m == -INFINITY) {   // nothing to draw from
        if (rank == 0 && t == 0) {
            p.tokens[r] = -1;
            if (p.logprobs) p.logprobs[r] = -INFINITY;
        }
        return;   // (nothing of a peer's is touched after the last exchange, here and below)
    }
    if (greedy) {   // the first warp that holds the largest logit finds its lowest index
        int owner = 0x7fffffff;
#pragma unroll
        for (int q = PER_LANE - 1; q >= 0; --q)
            if (wm[q] == m) owner = l * PER_LANE + q;
        if (static_cast<int>(__reduce_min_sync(0xffffffffu, owner)) / sub != me) return;
        int best = 0x7fffffff;
        for (int s = 0; s < steps && best == 0x7fffffff; ++s) {
            float x[8];
            ck.load(s * 256 + l * 8, x);
#pragma unroll
            for (int j = 7; j >= 0; --j)
                if (x[j] == m) best = s * 256 + l * 8 + j;
            best = __reduce_min_sync(0xffffffffu, best);
        }
        if (l == 0) {
            p.tokens[r] = first + best;
            if (p.logprobs) p.logprobs[r] = 0.f;
        }
        return;
    }

    SmpRow rw;
    rw.m = m;
    rw.ih = 1.f / temperature;
    rw.il = fmaf(-temperature, rw.ih, 1.f) * rw.ih;
    if (!(fabsf(rw.il) < INFINITY)) rw.il = 0.f;   // temperatures near the ends of the type's range
    if (!(m < INFINITY) || !(rw.ih < INFINITY)) {
        ck.only_max = true;
        ck.m = m;
        rw.m = 0.f;
        rw.ih = 1.f;
        rw.il = 0.f;
        temperature = 1.f;
#pragma unroll
        for (int q = 0; q < PER_LANE; ++q) wm[q] = wm[q] == m ? 0.f : -INFINITY;
        m = 0.f;
    }

    const bool by_count = SEARCH && top_k > 0 && top_k < p.V;
    const bool by_weight = SEARCH && top_p < 1.f;
    u64 w_min = 0;         // kept: weight at least w_min, ...
    if (min_p > 0.f) w_min = min_p >= 1.f ? SMP_ONE : smp_mul_floor(min_p, SMP_ONE, true);
    // ... and the cut: all logits with a key above cut_key, and the first cut_ties of those at it
    bool have_cut = false;
    uint32_t cut_key = 0, cut_ties = 0;
    u64 above = 0;         // the warp's kept weight above the cut, and its ties: formed
    uint32_t ties = 0;     // by the search (`summed`), or by a pass of their own
    bool summed = false;
    constexpr bool APART = SEARCH && sizeof(T) == 4;

    // writes the answer: token, its logit, and all kept weight
    auto answer = [&](long long token, float z, u64 total) {
        p.tokens[r] = token;
        if (p.logprobs) {
            constexpr float UNIT = 1.f / static_cast<float>(SMP_ONE);
            // log(total): the largest logit's weight is 1, so near 0 by log1p
            const float ls = total < 2 * SMP_ONE ? log1pf(static_cast<float>(total - SMP_ONE) * UNIT)
                                                 : logf(static_cast<float>(total) * UNIT);
            p.logprobs[r] = -smp_x(z, rw) - ls;
        }
    };
    // floor(u * total), u inside [0, 1): the token is the first whose cumulative weight exceeds it
    auto draw_target = [&](u64 total) -> u64 {
        if (!(u < 1.f)) return total - 1;
        return u > 0.f ? smp_mul_floor(u, total, false) : 0ull;
    };
    // the weight at which top-p ends, of `pool`
    auto share = [&](u64 pool) -> u64 {
        const u64 v = top_p > 0.f ? smp_mul_floor(top_p, pool, true) : 1ull;
        return v ? v : 1ull;
    };

    if (by_count || by_weight) {
        // A threshold with at least `want` logits at or above it, and rarely many more: the
        // want-th largest of the SMP_PARTS maxima of parts of the row, which go onto the list. Up to 32
        // of them are the lanes' maxima over PER_LANE parts, which every warp sorts for itself;
        // more are the parts' own, counted against one another. (top-k 50 with the list and without:
        // 64 x 128256 bf16 15.9 and 35.0 us, 1 x 32000 9.4 and 16.2.)
        constexpr int groups = 32;
        const int want = by_count ? top_k : groups - 1;           // (top-p: about 100 logits)
        bool use_list = want <= SMP_PARTS;
        float t0 = INFINITY;
        if (want <= groups) {
            float v = wm[0];
#pragma unroll
            for (int q = 1; q < PER_LANE; ++q) v = fmaxf(v, wm[q]);
            // bitonic sort, descending
#pragma unroll
            for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
                for (int j = k >> 1; j > 0; j >>= 1) {
                    const float o = __shfl_xor_sync(0xffffffffu, v, j);
                    const bool keep_max = ((l & j) == 0) == ((l & k) == 0);
                    v = keep_max ? fmaxf(v, o) : fminf(v, o);
                }
            t0 = __shfl_sync(0xffffffffu, v, want - 1);
            if (!by_count) {
                // Top-p of a flat row goes to the search at once: where the logits at the threshold, TAIL of
                // them, would outweigh what the largest may leave to the rest. (An estimate: either way
                // is right for every row, and every warp of the cluster forms the same one. With top-p 0.9
                // 64 x 128256 bf16 takes 60.4 us so and 74.6 with the list first; 1 x 32000 at a temperature
                // of 0.5, which the list holds, 10.8 and by the search 17.4.)
                constexpr float TAIL = 400.f;
                float e = __expf(-smp_x(v, rw));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
                use_list = !(TAIL * __expf(-smp_x(t0, rw)) * top_p > (1.f - top_p) * e);
            }
        } else if (use_list) {
#pragma unroll
            for (int q = 0; q < SMP_MAX_CLUSTER; ++q) {
                float v = sh.wmax[w * SMP_MAX_CLUSTER + q];   // every warp looks at its share of the parts
                if (ck.only_max) v = v == ck.m ? 0.f : -INFINITY;
                int more = 0, same = 0;
#pragma unroll
                for (int i = 0; i < PER_LANE; ++i) {
                    more += __popc(__ballot_sync(0xffffffffu, wm[i] > v));
                    same += __popc(__ballot_sync(0xffffffffu, wm[i] == v));
                }
                if (l == 0 && more < want && want <= more + same) sh.t0 = v;   // (all who write, write the same)
            }
        }
        if (t == 0) sh.listed = 0;
        __syncthreads();
        if (use_list) t0 = fmaxf(want <= groups ? t0 : sh.t0, -3.402823466e38f);   // (masked ones stay out)

        // one pass: the list, and (top-p alone) weights
        u64 pool = 0;        // weight of what top-k keeps
        if (use_list) {
            const bool weights = !by_count;
            u64 ws = 0, wl = 0;
            for (int s = 0; s < steps; ++s) {
                float x[8];
                ck.load(s * 256 + l * 8, x);
                if (weights) {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        u64 v0, v1;
                        smp_weight2(x[j], x[j + 1], rw, tabs, sh.tab, v0, v1);
                        ws += v0;
                        ws += v1;
                    }
                }
                bool any = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) any |= x[j] >= t0;
                if (__any_sync(0xffffffffu, any)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (!(x[j] >= t0)) continue;
                        const uint32_t at = atomicAdd(&sh.listed, 1u);
                        const uint32_t index = static_cast<uint32_t>(first) + s * 256 + l * 8 + j;
                        if (at < SMP_LIST_CTA) sh.list[at] = (static_cast<u64>(smp_key<T>(x[j])) << 32) | ~index;
                        if (weights) wl += smp_weight(x[j], rw, tabs, sh.tab);   // (few: cheaper than 8 kept)
                    }
                }
            }
            if (weights) {
                ws = warp_sum64(ws);
                wl = warp_sum64(wl);
            }
            if (l == 0) sh.part[w] = SmpSums{ws, wl, 0};
            __syncthreads();
            // lane k of warp 0 gives the CTA's sums to CTA k
            if (w == 0) {
                SmpSums o = l < SMP_WARPS ? sh.part[l] : SmpSums{0, 0, 0};
                o.w = warp_sum64(o.w);
                o.wlist = warp_sum64(o.wlist);
                o.list = sh.listed;
                if (l < static_cast<int>(cl)) {
                    const uint32_t at = map_to_rank(&sh.sums[rank], l);
                    auto hi = [](u64 v) { return static_cast<uint32_t>(v >> 32); };
                    auto lo = [](u64 v) { return static_cast<uint32_t>(v); };
                    st_cluster_v4(at, lo(o.w), hi(o.w), lo(o.wlist), hi(o.wlist));
                    st_cluster_v4(at + 16, o.list, 0u, 0u, 0u);
                }
            }
            cluster_sync_all();
            SmpSums sum = {0, 0, 0};
            bool over = false;
            for (uint32_t k = 0; k < cl; ++k) {
                const SmpSums &o = sh.sums[k];
                sum.w += o.w;
                sum.wlist += o.wlist;
                sum.list += o.list;
                over |= o.list > SMP_LIST_CTA;
            }
            // with top-k the list holds all that it keeps; with top-p alone, all that p keeps if it
            // weighs enough
            if (!over && sum.list <= SMP_LIST && (by_count || sum.wlist >= share(sum.w))) {
                if (rank == 0) {
                    // thread i: entry i of the list
                    const int n_list = static_cast<int>(sum.list);
                    u64 c = 0, wt = 0;
                    float z = 0.f;
                    if (t < n_list) {
                        int at = t;
                        uint32_t k = 0;
                        while (at >= static_cast<int>(sh.sums[k].list)) at -= static_cast<int>(sh.sums[k++].list);
                        c = ld_cluster_u64(map_to_rank(&sh.list[at], k));
                        z = smp_unkey<T>(static_cast<uint32_t>(c >> 32));
                        wt = smp_weight(z, rw, tabs, sh.tab);
                        sh.all[t] = c;
                        sh.allw[t] = wt;
                    }
                    __syncthreads();
                    int before = 0;    // entries and weight before this one in the order
                    u64 before_w = 0;
                    if (t < n_list)
                        for (int j = 0; j < n_list; ++j)
                            if (sh.all[j] > c) {
                                ++before;
                                before_w += sh.allw[j];
                            }
                    // sum over the CTA of one value per thread
                    auto block_sum = [&](u64 v) {
                        v = warp_sum64(v);
                        __syncthreads();
                        if (l == 0) sh.wsum[w] = v;
                        __syncthreads();
                        u64 a = 0;
                        for (int k = 0; k < SMP_WARPS; ++k) a += sh.wsum[k];
                        return a;
                    };
                    bool keep = t < n_list && (!by_count || before < top_k);
                    if (by_weight) {
                        const u64 end = share(by_count ? block_sum(keep ? wt : 0ull) : sum.w);
                        keep = keep && before_w < end;
                    }
                    keep = keep && wt >= w_min;
                    const u64 total = block_sum(keep ? wt : 0ull);   // (all have read sh.allw)
                    if (t < n_list) sh.allw[t] = keep ? wt : 0ull;
                    __syncthreads();
                    const u64 target = draw_target(total);
                    const uint32_t index = ~static_cast<uint32_t>(c);
                    if (keep) {
                        u64 upto = wt;   // kept weight up to and including this index
                        for (int j = 0; j < n_list; ++j)
                            if (~static_cast<uint32_t>(sh.all[j]) < index) upto += sh.allw[j];
                        if (upto > target && upto - wt <= target) answer(index, z, total);
                    }
                }
                cluster_sync_all();   // rank 0 has read the peers' lists
                return;
            }
        }
        // ---- the general search: a histogram of x, then of the keys in the bin that holds the cut
        int hb = 0;   // histogram in use
        auto clear = [&]() {
            for (int k = t; k < 4 * SMP_BINS; k += SMP_THREADS) (&sh.hist[hb][0][0])[k] = 0u;
            __syncthreads();
        };
        // totals over the cluster of the histogram just filled; exclusive prefixes over
        // its bins into (pc, pw). one_key: each bin holds the logits of one key, khi less the
        // bin's number, and only counts were added: their weight is the key's times the count
        auto totals = [&](uint32_t *pc, u64 *pw, uint32_t *tot_c, u64 *tot_w, bool one_key, uint32_t khi) {
            cluster_sync_all();
            uint32_t c = 0;
            u64 wt = 0;
            if (t < SMP_BINS) {
                // (all loads are under way before the first is used)
                uint32_t h[4][SMP_MAX_CLUSTER];
#pragma unroll
                for (uint32_t k = 0; k < SMP_MAX_CLUSTER; ++k) {
                    h[0][k] = h[1][k] = h[2][k] = h[3][k] = 0u;
                    if (k >= cl) continue;
                    const uint32_t at = map_to_rank(&sh.hist[hb][0][t], k);
                    if (by_count || one_key) h[0][k] = ld_cluster_u32(at);
                    if (by_weight && !one_key) {
                        h[1][k] = ld_cluster_u32(at + 4 * SMP_BINS);
                        h[2][k] = ld_cluster_u32(at + 8 * SMP_BINS);
                        h[3][k] = ld_cluster_u32(at + 12 * SMP_BINS);
                    }
                }
                u64 l0 = 0, l1 = 0, l2 = 0;
#pragma unroll
                for (uint32_t k = 0; k < SMP_MAX_CLUSTER; ++k) {
                    c += h[0][k];
                    l0 += h[1][k];
                    l1 += h[2][k];
                    l2 += h[3][k];
                }
                wt = l0 + (l1 << SMP_LIMB) + (l2 << (2 * SMP_LIMB));
                if (one_key && by_weight && c)
                    wt = c * smp_weight(smp_unkey<T>(khi - static_cast<uint32_t>(t)), rw, tabs, sh.tab);
                uint32_t ci = c;
                u64 wi = wt;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t c2 = __shfl_up_sync(0xffffffffu, ci, o);
                    const u64 w2 = shfl_up64(wi, o);
                    if (l >= o) {
                        ci += c2;
                        wi += w2;
                    }
                }
                if (l == 31) {
                    sh.csum[w] = ci;
                    sh.wsum[w] = wi;
                }
                pc[t] = ci - c;
                pw[t] = wi - wt;
            }
            __syncthreads();
            uint32_t cb = 0;
            u64 wb = 0;
            for (int k = 0; k < SMP_BINS / 32; ++k) {
                if (k == w && t < SMP_BINS) {
                    pc[t] += cb;
                    pw[t] += wb;
                }
                cb += sh.csum[k];
                wb += sh.wsum[k];
            }
            *tot_c = cb;
            *tot_w = wb;
            __syncthreads();
            hb ^= 1;
        };
        // the bin in which `target` (a count, or a weight) is reached
        auto find = [&](const uint32_t *pc, const u64 *pw, uint32_t tot_c, u64 tot_w, bool count,
                        u64 target) {
            if (t < SMP_BINS) {
                const uint32_t c0 = pc[t], c1 = t + 1 < SMP_BINS ? pc[t + 1] : tot_c;
                const u64 w0 = pw[t], w1 = t + 1 < SMP_BINS ? pw[t + 1] : tot_w;
                const u64 a = count ? c0 : w0, b = count ? c1 : w1;
                // (the sums are exact, so one bin always fits; the ends keep any target in range)
                if ((a < target && target <= b) || (t == 0 && target == 0) || (t == SMP_BINS - 1 && b < target)) {
                    sh.bin = t;
                    sh.bc = c0;
                    sh.bw = w0;
                }
            }
            __syncthreads();
        };

        // first level: bins of x
        uint32_t tot_c = 0;
        u64 tot_w = 0;
        // bin: the lesser of two lines in x, rounded to nearest by adding SMP_ROUND (a conversion
        // runs at a fraction of the rate)
        constexpr float NEAR = SMP_BINS / 2 / SMP_X_MID, FAR = (SMP_BINS / 2 - 1) / (SMP_X_END - SMP_X_MID);
        constexpr float FAR_0 = SMP_BINS / 2 - SMP_X_MID * FAR;
        auto bin_of = [&](float z) {
            const float xx = smp_x(z, rw);
            const float y = fminf(xx * NEAR, fmaf(xx, FAR, FAR_0));
            return xx < SMP_X_END ? __float_as_int(y + SMP_ROUND) & (SMP_BINS - 1) : -1;
        };
        auto bin_start = [&](int b) {
            const float y = static_cast<float>(b) - 0.5f;
            return fmaxf(y < SMP_BINS / 2 ? y / NEAR : (y - FAR_0) / FAR, 0.f);
        };
        auto first_level = [&]() {
            clear();
            for (int s = 0; s < steps; ++s) {
                float x[8];
                ck.load(s * 256 + l * 8, x);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    u64 v0 = 0, v1 = 0;
                    if (by_weight) smp_weight2(x[j], x[j + 1], rw, tabs, sh.tab, v0, v1);
                    const int b0 = bin_of(x[j]), b1 = bin_of(x[j + 1]);
                    if (b0 >= 0) smp_hist_add(sh.hist[hb], b0, by_count, by_weight, v0);
                    if (b1 >= 0) smp_hist_add(sh.hist[hb], b1, by_count, by_weight, v1);
                }
            }
            totals(sh.l0c, sh.l0w, &tot_c, &tot_w, false, 0u);
        };

        // the key and the number of equal logits at which `target` is reached
        auto search = [&](bool count, u64 target, uint32_t *key, uint32_t *ties, u64 *kept_w) {
            // keys that include those of x from near_x to far_x, with room for the roundings
            uint32_t klo, khi;
            auto key_range = [&](float near_x, float far_x) {
                klo = smp_key<T>(-3.402823466e38f);
                khi = smp_key<T>(m);
                const float room = (fabsf(m) + far_x * temperature) * 1e-6f + 1e-37f;
                const float zhi = m - near_x * temperature + room, zlo = m - far_x * temperature - room;
                if (zhi < m) khi = smp_key<T>(zhi);
                if (zlo > -3e38f) klo = smp_key<T>(zlo);
            };
            find(sh.l0c, sh.l0w, tot_c, tot_w, count, target);
            const int b0 = sh.bin;
            uint32_t base_c = sh.bc;
            u64 base_w = sh.bw;
            __syncthreads();
            key_range(bin_start(b0), bin_start(b0 + 1));
            // fp32 and the only search: one pass sums what lies before the bin and keeps the bin's logits
            // apart, on which the rest of the search runs. (Top-p 0.9, with and without: 256 x 128256 fp32
            // 225 and 260 us; bf16, whose bins rarely need a second histogram, 64 x 128256 64.6 and 61.2.)
            int n_bin = 0;
            if constexpr (APART) {
                const bool last = b0 + 1 == SMP_BINS;   // logits in the bin: counted, or its weight over that of one
                const float inside = count ? static_cast<float>((last ? tot_c : sh.l0c[b0 + 1]) - base_c)
                                           : static_cast<float>((last ? tot_w : sh.l0w[b0 + 1]) - base_w) / SMP_ONE *
                                                 __expf(0.5f * (bin_start(b0) + bin_start(b0 + 1)));
                if (by_count != by_weight && inside < 0.9f * SMP_BIN_CTA * cl) {
                    if (t == 0) sh.listed = 0;
                    if (t < SMP_WARPS) {
                        sh.bin_w[t] = 0;
                        sh.bin_t[t] = 0;
                    }
                    __syncthreads();
                    for (int s = 0; s < steps; ++s) {
                        float x[8];
                        ck.load(s * 256 + l * 8, x);
                        uint32_t before = 0, in = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int bin = bin_of(x[j]);
                            if (bin >= 0 && bin < b0) before |= 1u << j;
                            if (bin == b0) in |= 1u << j;
                        }
                        if (__any_sync(0xffffffffu, before != 0)) {
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                u64 v0, v1;
                                smp_weight2(x[j], x[j + 1], rw, tabs, sh.tab, v0, v1);
                                if (!(before >> j & 1u) || v0 < w_min) v0 = 0ull;
                                if (!(before >> j & 2u) || v1 < w_min) v1 = 0ull;
                                above += v0;
                                above += v1;
                            }
                        }
                        if (in) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (!(in >> j & 1u)) continue;
                                const uint32_t at = atomicAdd(&sh.listed, 1u);
                                if (at < SMP_BIN_CTA) {
                                    sh.bin_key[at] = smp_key<T>(x[j]);
                                    sh.bin_warp[at] = static_cast<uint8_t>(w);
                                }
                            }
                        }
                    }
                    __syncthreads();
                    summed = sh.listed <= SMP_BIN_CTA;
                    if (!summed) above = 0;
                }
                if (summed) n_bin = static_cast<int>(sh.listed);
            }
            for (int level = 0; klo != khi && level < 4; ++level) {   // 8 bits of the key at a time
                const int bits = 32 - __clz(khi - klo);
                const int shift = bits > 8 ? bits - 8 : 0;
                const float zlo = smp_unkey<T>(klo), zhi = smp_unkey<T>(khi);
                clear();
                auto add = [&](uint32_t k, float z) {
                    if (shift == 0) atomicAdd(&sh.hist[hb][0][khi - k], 1u);
                    else
                        smp_hist_add(sh.hist[hb], static_cast<int>((khi - k) >> shift), by_count, by_weight,
                                     by_weight ? smp_weight(z, rw, tabs, sh.tab) : 0ull);
                };
                for (int i = t; APART && i < n_bin; i += SMP_THREADS) {
                    const uint32_t k = sh.bin_key[i];
                    if (k >= klo && k <= khi) add(k, smp_unkey<T>(k));
                }
                for (int s = 0; s < (APART && summed ? 0 : steps); ++s) {
                    float x[8];
                    bool any = false;
                    ck.load(s * 256 + l * 8, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) any |= x[j] >= zlo && x[j] <= zhi;
                    if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (!(x[j] >= zlo && x[j] <= zhi)) continue;
                        const uint32_t k = smp_key<T>(x[j]);
                        const int in = bin_of(x[j]);
                        if (!(k >= klo && k <= khi && in == b0)) continue;
                        add(k, x[j]);
                    }
                }
                uint32_t tc;
                u64 tw;
                totals(sh.rc, sh.rw, &tc, &tw, shift == 0, khi);
                find(sh.rc, sh.rw, tc, tw, count, target - (count ? static_cast<u64>(base_c) : base_w));
                const uint32_t b = static_cast<uint32_t>(sh.bin);
                base_c += sh.bc;
                base_w += sh.bw;
                khi -= min(b << shift, khi - klo);
                const uint32_t width = (1u << shift) - 1u;
                klo = khi - klo > width ? khi - width : klo;
                __syncthreads();
            }
            if constexpr (APART) {
                for (int i = t; i < n_bin; i += SMP_THREADS) {   // the bin's share of the warps' sums
                    const uint32_t k = sh.bin_key[i];
                    if (k > klo) {
                        const u64 v = smp_weight(smp_unkey<T>(k), rw, tabs, sh.tab);
                        if (v >= w_min) atomicAdd(&sh.bin_w[sh.bin_warp[i]], v);
                    } else if (k == klo) {
                        atomicAdd(&sh.bin_t[sh.bin_warp[i]], 1u);
                    }
                }
                __syncthreads();
            }
            *key = klo;
            const u64 one = by_weight ? smp_weight(smp_unkey<T>(klo), rw, tabs, sh.tab) : 1ull;
            *ties = count ? static_cast<uint32_t>(target) - base_c
                          : static_cast<uint32_t>((target - base_w + one - 1) / one);
            *kept_w = base_w + static_cast<u64>(*ties) * one;
        };

        first_level();
        pool = tot_w;
        if (by_count && static_cast<uint32_t>(top_k) < tot_c) {
            search(true, static_cast<u64>(top_k), &cut_key, &cut_ties, &pool);
            have_cut = true;
        }
        if (by_weight) {
            uint32_t key, ties;
            u64 kept;
            search(false, share(pool), &key, &ties, &kept);
            if (!have_cut || key > cut_key || (key == cut_key && ties < cut_ties)) {
                cut_key = key;
                cut_ties = ties;
            }
            have_cut = true;
        }
    }

    const float cut = have_cut ? smp_unkey<T>(cut_key) : -INFINITY;
    const u64 tie_w0 = have_cut ? smp_weight(cut, rw, tabs, sh.tab) : 0ull;
    const u64 tie_w = tie_w0 >= w_min ? tie_w0 : 0ull;
    // weights above the cut of 8 logits
    auto kept_weights = [&](const float (&x)[8], u64 (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) smp_weight2(x[j], x[j + 1], rw, tabs, sh.tab, v[j], v[j + 1]);
        if (have_cut) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (!(x[j] > cut)) v[j] = 0ull;
        }
        if (w_min) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (v[j] < w_min) v[j] = 0ull;
        }
    };

    // sums of every warp of the cluster, in index order
    for (int s = 0; s < (APART && summed ? 0 : steps); ++s) {
        float x[8];
        ck.load(s * 256 + l * 8, x);
        if (have_cut) {
            bool any = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                any |= x[j] > cut;
                ties += x[j] == cut ? 1u : 0u;
            }
            if (!__any_sync(0xffffffffu, any)) continue;
        }
        u64 v[8];
        kept_weights(x, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) above += v[j];
    }
    above = warp_sum64(above);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (APART && summed) {
        above += sh.bin_w[w];
        ties = sh.bin_t[w];
    }
    if (l < static_cast<int>(cl))
        st_cluster_v4(map_to_rank(&sh.wslot[rank * SMP_WARPS + w], l), static_cast<uint32_t>(above),
                      static_cast<uint32_t>(above >> 32), ties, 0u);
    cluster_sync_all();

    // every warp sums all warps' entries: 4 per lane, in order
    u64 ew[PER_LANE];
    uint32_t et[PER_LANE], lane_t = 0;
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        const int e = l * PER_LANE + q;
        const uint4 v = e < entries ? sh.wslot[e] : make_uint4(0u, 0u, 0u, 0u);
        ew[q] = static_cast<u64>(v.x) | (static_cast<u64>(v.y) << 32);
        et[q] = v.z;
        lane_t += v.z;
    }
    uint32_t before_t = lane_t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, before_t, o);
        if (l >= o) before_t += v;
    }
    before_t -= lane_t;
    const uint32_t lane_t0 = before_t;
    u64 lane_w = 0;
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        const uint32_t room = before_t < cut_ties ? cut_ties - before_t : 0u;
        ew[q] += static_cast<u64>(et[q] < room ? et[q] : room) * tie_w;
        lane_w += ew[q];
        before_t += et[q];
    }
    u64 incl = lane_w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = shfl_up64(incl, o);
        if (l >= o) incl += v;
    }
    const u64 total = __shfl_sync(0xffffffffu, incl, 31);

    // The first index whose cumulative weight exceeds u * total: the warp in whose part it lies, ...
    const u64 target = draw_target(total);
    const int lane = __ffs(__ballot_sync(0xffffffffu, incl > target)) - 1;   // (always one: total > target)
    u64 run = incl - lane_w;   // kept weight and ties before the part
    uint32_t seen = lane_t0;
    int part = l * PER_LANE;
    bool passed = true;
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        passed = passed && run + ew[q] <= target;
        if (passed) {
            run += ew[q];
            seen += et[q];
            ++part;
        }
    }
    run = __shfl_sync(0xffffffffu, run, lane);
    seen = __shfl_sync(0xffffffffu, seen, lane);
    part = __shfl_sync(0xffffffffu, part, lane);
    if (part / SMP_WARPS != static_cast<int>(rank)) return;   // (nothing of a peer's is touched after the exchange)
    // ... the sweep of that part, whose sums the CTA's warps form side by side (by one
    // warp alone 64 x 128256 bf16 takes 21.7 us instead of 18.1), ...
    {
        const long long first = static_cast<long long>(part) * chunk;
        const long long left = p.V - first;
        ck.n = left <= 0 ? 0 : left < chunk ? static_cast<int>(left) : chunk;
        if constexpr (SMEM) {
            ck.p = reinterpret_cast<const T *>(smp_dyn) + static_cast<size_t>(part % SMP_WARPS) * chunk;
        } else {
            ck.p = static_cast<const T *>(p.Z) + r * p.ld + (ck.n > 0 ? first : 0);
            ck.aligned = (reinterpret_cast<uintptr_t>(ck.p) & 15u) == 0;
        }
        const int sweeps = (ck.n + 255) / 256;
        int sweep = 0;
        if (sweeps > 1) {
            for (int s = w; s < sweeps; s += SMP_WARPS) {
                float x[8];
                u64 v[8], sum = 0;
                uint32_t same = 0;
                ck.load(s * 256 + l * 8, x);
                kept_weights(x, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum += v[j];
                    same += have_cut && x[j] == cut ? 1u : 0u;
                }
                sum = warp_sum64(sum);
                if (have_cut) same = __reduce_add_sync(0xffffffffu, same);
                if (l == 0) {
                    sh.sweep_w[s] = sum;
                    sh.sweep_t[s] = same;
                }
            }
            __syncthreads();
            if (w != 0) return;
            u64 sum = l < sweeps ? sh.sweep_w[l] : 0ull;
            const uint32_t same = l < sweeps ? sh.sweep_t[l] : 0u;
            uint32_t upto = same;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t c = __shfl_up_sync(0xffffffffu, upto, o);
                if (l >= o) upto += c;
            }
            const uint32_t before = seen + upto - same;
            const uint32_t room = before < cut_ties ? cut_ties - before : 0u;
            sum += static_cast<u64>(same < room ? same : room) * tie_w;
            u64 in = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 c = shfl_up64(in, o);
                if (l >= o) in += c;
            }
            // (one is always found, unless Z changes meanwhile)
            sweep = max(__ffs(__ballot_sync(0xffffffffu, run + in > target)) - 1, 0);
            run += __shfl_sync(0xffffffffu, in - sum, sweep);
            seen = __shfl_sync(0xffffffffu, before, sweep);
        } else if (w != 0) {
            return;
        }
        // ... and the index
        const int i = sweep * 256 + l * 8;
        float x[8];
        u64 v[8];
        uint32_t tmask = 0;
        ck.load(i, x);
        kept_weights(x, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (have_cut && x[j] == cut) tmask |= 1u << j;
        const uint32_t tl = __popc(tmask);
        uint32_t tb = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t c = __shfl_up_sync(0xffffffffu, tb, o);
            if (l >= o) tb += c;
        }
        uint32_t mine_seen = seen + tb - tl;
        u64 sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (tmask >> j & 1u) v[j] = mine_seen++ < cut_ties ? tie_w : 0ull;
            sum += v[j];
        }
        u64 in = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 c = shfl_up64(in, o);
            if (l >= o) in += c;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + in > target);
        if (l == __ffs(hit) - 1) {
            u64 c = run + in - sum;
            int at = 0;
            float z = x[0];
            bool found = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c += v[j];
                if (!found && c > target) {
                    found = true;
                    at = j;
                    z = x[j];
                }
            }
            answer(first + i + at, z, total);
        }
    }
}

using SampleKernel = void (*)(const SampleParams, const SampleTables, const int);

template <typename T> SampleKernel sample_kernel_of(bool smem, bool search) {
    if (smem) return search ? lce_sample_kernel<T, true, true> : lce_sample_kernel<T, true, false>;
    return search ? lce_sample_kernel<T, false, true> : lce_sample_kernel<T, false, false>;
}
SampleKernel sample_kernel(int dtype, bool smem, bool search) {
    if (dtype == CE_FP32) return sample_kernel_of<float>(smem, search);
    if (dtype == CE_FP16) return sample_kernel_of<__half>(smem, search);
    return sample_kernel_of<__nv_bfloat16>(smem, search);
}

constexpr int SMP_MAX_DYN = 160 * 1024;   // a CTA's logits; the rest of its shared memory is static
constexpr int SMP_TWO_DYN = 83 * 1024;    // the same when two CTAs share an SM
static_assert(SMP_MAX_V <= static_cast<long long>(SMP_MAX_CTA) * SMP_MAX_CLUSTER, "the longest row must fit");

}  // namespace

cudaError_t sample_set_attributes() {
    for (int dt = CE_BF16; dt <= CE_FP16; ++dt) {
        for (int search = 0; search < 2; ++search) {
            const cudaError_t e = cudaFuncSetAttribute(
                sample_kernel(dt, true, search != 0), cudaFuncAttributeMaxDynamicSharedMemorySize, SMP_MAX_DYN);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

cudaError_t launch_sample(const SampleParams &p, int sms, cudaStream_t s) {
    if (p.N <= 0) return cudaSuccess;
    static const SampleTables tabs = make_sample_tables();
    const long long elem = p.dtype == CE_FP32 ? 4 : 2;
    const bool search = p.top_k || p.top_p || p.top_k_all > 0 || p.top_p_all < 1.f;
    // CTAs per row: of 1, 2, 4 and 8 the one with the least estimated time (us). A CTA takes 0.235 us
    // per 1000 logits and a start and exchanges that grow with the cluster; those of an SM follow one
    // another, but two at once hide the latency that a single one shows (30 %). Rows that do not
    // fit into shared memory twice per SM (once, where one CTA per SM is all there is) are read again
    // from L2: 5 % more, and 30 % if the rows under way are more than it holds. Measured, us, CTAs per row
    // 1 / 2 / 4 / 8 (*: read again):
    //   1 x 32000 bf16            14.7   10.3    8.7    6.2
    //   64 x 128256 bf16          60     28.5   24.6   29.3   (32 x 50257 fp16: 25.5 16.8 12.1 12.8)
    //   100 x 32000 fp32          16.6   15.4   19.4   22.8
    //   160 x 128256 fp32         75.7*  61.8*  53.9*  65.5
    //   256 x 128256 bf16         78.0*  74.8*  72.1   90.3
    //   256 x 128256 fp32         90.6*  79.7*  78.5*  100.1
    //   512 x 50257 fp16          84.5*  74.0   96.9   146
    //   600 x 32000 bf16          41.9   49.1   73.7   122
    //   1024 x 128256 bf16        226*   228*   258    342
    auto chunk_of = [&](int c) { return ((p.V + c * SMP_WARPS - 1) / (c * SMP_WARPS) + 7) / 8 * 8; };
    constexpr double PER_LOGIT = 0.235e-3, PER_CTA[4] = {0.9, 0.9, 1.6, 2.5}, L2_ROWS = 96e6;
    int cl = 1;
    bool smem = false;
    double best = 1e30;
    for (int k = 0; k < 4; ++k) {
        const int c = 1 << k;
        if (k > 0 && chunk_of(c / 2) <= 256) break;   // a warp of a smaller cluster has one sweep
        const double bytes = static_cast<double>(chunk_of(c)) * SMP_WARPS * elem;
        if (bytes / elem > SMP_MAX_CTA) continue;
        const long long per_sm = (p.N * c + sms - 1) / sms;
        const bool fits = bytes <= (per_sm == 1 ? SMP_MAX_DYN : SMP_TWO_DYN);
        const double logits = static_cast<double>(p.V) / c * PER_LOGIT;
        double us = per_sm == 1 ? 1.3 * logits : per_sm * (logits + PER_CTA[k]);
        if (!fits) {
            const double rows = static_cast<double>(std::min<long long>(p.N * c, 2 * sms)) / c;
            us *= rows * p.V * elem > L2_ROWS ? 1.3 : 1.05;
        }
        if (us < best) {
            best = us;
            cl = c;
            smem = fits;
        }
    }
    const long long chunk = chunk_of(cl);
    const long long bytes = chunk * SMP_WARPS * elem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cl;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.N * cl));
    cfg.blockDim = dim3(SMP_THREADS);
    cfg.dynamicSmemBytes = smem ? static_cast<size_t>(bytes) : 0;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel(p.dtype, smem, search), p, tabs, static_cast<int>(chunk));
}

}  // namespace lce
