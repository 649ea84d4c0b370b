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
// to a relative error of about 2^-32: the sum of border displacements over a row
// of 2^17 equally likely tokens is about 1e-8, which bounds the chance that u falls
// on the wrong side of one. An fp32 softmax would put it at about 1e-2.
//
// Bound: one read of the logits. A cluster of CTAs holds a row in shared memory,
// so every later pass (the search for the cut, the sums, the draw) stays on chip; the
// CTAs exchange maxima, histograms and sums through distributed shared memory. Rows
// longer than the cluster's shared memory are read again from L2 instead.
#include <cmath>

#include "lce_internal.h"
#include "lce_ptx.cuh"

namespace lce {

constexpr int SMP_THREADS = 512;
constexpr int SMP_WARPS = SMP_THREADS / 32;
constexpr int SMP_MAX_CLUSTER = 8;
constexpr int SMP_BINS = 256;
constexpr int SMP_ONE_SHIFT = 43;                    // weight of the largest logit: 2^43
constexpr int SMP_TAB_SHIFT = 50;                    // the exponential's table is kept in units of 2^-50
constexpr float SMP_X_END = 31.f;                    // exp(-31) < 2^-44 rounds to weight 0
constexpr float SMP_BINS_PER_UNIT = 8.f;             // 31 * 8 = 248 bins of x
constexpr int SMP_LIMB = 15;                         // bits per limb of a weight: 2^17 limbs fit 32 bits

// Constants of the exponential, from their definitions on the host.
SampleTables make_sample_tables() {
    SampleTables t;
    const double ln2 = std::log(2.0);
    for (int j = 0; j < 64; ++j) {
        const double v = std::exp2(-j / 64.0);
        t.fix[j] = static_cast<unsigned long long>(std::nearbyint(std::ldexp(v, SMP_TAB_SHIFT)));
        t.flt[j] = static_cast<float>(v);
    }
    // ln(2) / 64 in three parts: 12 bits (its product with a whole number below
    // 2^12 is exact), 24 bits, and the rest
    const double step = ln2 / 64.0;
    int e;
    std::frexp(step, &e);
    const double ulp = std::ldexp(1.0, e - 12);
    const double c1 = std::floor(step / ulp) * ulp;
    t.c1 = static_cast<float>(c1);
    t.c2 = static_cast<float>(step - c1);
    t.c3 = static_cast<float>(step - c1 - static_cast<double>(t.c2));
    t.inv = static_cast<float>(64.0 / ln2);
    return t;
}

namespace {

typedef unsigned long long u64;

// ------------------------------------------------------------------ logits in vectors of 8

__device__ __forceinline__ float smp_clean(float x) {
    // NaN becomes -infinity (never drawn), -0 becomes +0 (equal to it in the order)
    return fmaxf(x, -INFINITY) + 0.f;
}
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
__device__ __forceinline__ uint32_t smp_pack2(float a, float b, const __nv_bfloat16 *) {
    return (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
}
__device__ __forceinline__ uint32_t smp_pack2(float a, float b, const __half *) {
    const __half2 h = __floats2half2_rn(a, b);   // exact: the values are halves
    return *reinterpret_cast<const uint32_t *>(&h);
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
template <typename T> __device__ __forceinline__ void smp_store_vec(T *p, const float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        const T *t = nullptr;
        *reinterpret_cast<uint4 *>(p) = make_uint4(smp_pack2(x[0], x[1], t), smp_pack2(x[2], x[3], t),
                                                   smp_pack2(x[4], x[5], t), smp_pack2(x[6], x[7], t));
    }
}
// 8 cleaned logits from global memory; those past `n` are -infinity.
template <typename T>
__device__ __forceinline__ void smp_load_global(const T *p, int n, bool aligned, float (&x)[8]) {
    if (aligned && n >= 8) {
        smp_load_vec<T>(p, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = smp_clean(x[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < n ? smp_clean(static_cast<float>(p[j])) : -INFINITY;
    }
}

// Order-preserving whole number of a logit. 16-bit types: the 32-bit pattern's low
// bits, which are the same for all values of the type and sign, are dropped.
template <typename T> struct SmpKey;
template <> struct SmpKey<__nv_bfloat16> { static constexpr int DROP = 16; };
template <> struct SmpKey<__half> { static constexpr int DROP = 13; };
template <> struct SmpKey<float> { static constexpr int DROP = 0; };

template <typename T> __device__ __forceinline__ uint32_t smp_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return (b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) >> SmpKey<T>::DROP;
}
template <typename T> __device__ __forceinline__ float smp_unkey(uint32_t key) {
    constexpr int DROP = SmpKey<T>::DROP;
    uint32_t b = key << DROP;
    if (b >> 31) return __uint_as_float(b ^ 0x80000000u);
    return __uint_as_float((~b) & ~((1u << DROP) - 1u));
}

// ------------------------------------------------------------------ weights

struct SmpTab {            // in shared memory
    u64 fix[64];
    float flt[64];
};
struct SmpRow {
    float m, ih, il;       // largest logit; 1 / temperature in two parts
    float c1, c2, c3, inv;
};

// x = (m - z) / temperature, rounded: the same monotone function wherever it is used.
__device__ __forceinline__ float smp_x(float z, const SmpRow &r) {
    return z == r.m ? 0.f : (r.m - z) * r.ih;
}

// exp(-(m - z) / temperature) in units of 2^-43. x is carried in two floats (xh + xl);
// x = n ln(2) / 64 + rr, exp(-x) = 2^-(n / 64) * (1 + q) with q = exp(-rr) - 1,
// |rr| < 0.0055; the table's part is exact to 2^-51, T * q to 2^-32.
__device__ __forceinline__ u64 smp_weight(float z, const SmpRow &r, const SmpTab &tab) {
    if (z == r.m) return 1ull << SMP_ONE_SHIFT;
    const float d = r.m - z;
    const float xh = d * r.ih;
    if (!(xh < SMP_X_END)) return 0ull;
    const float bb = d - r.m;
    const float dl = (r.m - (d - bb)) - (z + bb);      // d + dl = m - z exactly
    float xl = fmaf(d, r.ih, -xh);
    xl = fmaf(d, r.il, xl);
    xl = fmaf(dl, r.ih, xl);
    const float nf = rintf(xh * r.inv);
    const int n = static_cast<int>(nf);
    float rr = fmaf(-nf, r.c1, xh);                    // exact
    xl = fmaf(-nf, r.c3, xl);
    rr = fmaf(-nf, r.c2, rr) + xl;
    const float q = rr * fmaf(rr, fmaf(rr, fmaf(rr, 1.f / 24.f, -1.f / 6.f), 0.5f), -1.f);
    const int j = n & 63, e = n >> 6;
    const int f = __float2int_rn(tab.flt[j] * q * 274877906944.f);   // T q in units of 2^-38
    const long long w = static_cast<long long>(tab.fix[j]) +
                        (static_cast<long long>(f) << (SMP_TAB_SHIFT - 38));
    const int s = SMP_TAB_SHIFT - SMP_ONE_SHIFT + e;   // 7 .. 52
    return (static_cast<u64>(w) + (1ull << (s - 1))) >> s;
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
__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
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

struct SmpShared {
    uint4 hist[2][SMP_BINS];              // {count, three limbs of the weight}; read by the peers
    uint4 slot[2][SMP_MAX_CLUSTER];       // one exchanged value per CTA
    uint4 wslot[SMP_MAX_CLUSTER * SMP_WARPS];   // per warp of the cluster: sum above the cut, ties
    u64 l0w[SMP_BINS], rw[SMP_BINS];      // weight before each bin: first level, refinement
    uint32_t l0c[SMP_BINS], rc[SMP_BINS]; // count before each bin
    u64 wsum[SMP_BINS / 32];
    uint32_t csum[SMP_BINS / 32];
    u64 bw, bwin;                         // the bin found: weight before it, in it
    uint32_t bc, bcin;
    int bin;
    float red[SMP_WARPS];
    uint32_t redlo[SMP_WARPS], redhi[SMP_WARPS];
    SmpTab tab;
};

// The warp's part of the row: `n` logits from index `first` on, in shared memory
// (cleaned, filled up to a multiple of 8 with -infinity) or in global memory.
template <typename T, bool SMEM> struct SmpChunk {
    const T *p;
    int n;
    bool aligned;
    __device__ __forceinline__ void load(int i, float (&x)[8]) const {
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

// Adds to the histogram; `b` < 0: nothing. A warp whose lanes all hit one bin (equal
// logits) adds once.
template <bool WEIGHTS>
__device__ __forceinline__ void smp_hist_add(uint4 *hist, int b, u64 w, int lane) {
    const int b0 = __shfl_sync(0xffffffffu, b, 0);
    if (__all_sync(0xffffffffu, b == b0)) {
        if (b0 < 0) return;
        if constexpr (WEIGHTS) {
            constexpr uint32_t M = (1u << SMP_LIMB) - 1u;
            const uint32_t s0 = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w) & M);
            const uint32_t s1 =
                __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w >> SMP_LIMB) & M);
            const uint32_t s2 =
                __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w >> (2 * SMP_LIMB)));
            if (lane == 0) {
                atomicAdd(&hist[b0].y, s0);
                atomicAdd(&hist[b0].z, s1);
                atomicAdd(&hist[b0].w, s2);
            }
        }
        if (lane == 0) atomicAdd(&hist[b0].x, 32u);
        return;
    }
    if (b < 0) return;
    atomicAdd(&hist[b].x, 1u);
    if constexpr (WEIGHTS) {
        constexpr uint32_t M = (1u << SMP_LIMB) - 1u;
        atomicAdd(&hist[b].y, static_cast<uint32_t>(w) & M);
        atomicAdd(&hist[b].z, static_cast<uint32_t>(w >> SMP_LIMB) & M);
        atomicAdd(&hist[b].w, static_cast<uint32_t>(w >> (2 * SMP_LIMB)));
    }
}

template <typename T, bool SMEM>
__global__ void __launch_bounds__(SMP_THREADS)
    lce_sample_kernel(const SampleParams p, const __grid_constant__ SampleTables tabs, const int chunk) {
    extern __shared__ __align__(128) uint8_t smp_dyn[];
    __shared__ SmpShared sh;
    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    const uint32_t rank = cluster_ctarank(), cl = smp_cluster_size();
    const long long r = blockIdx.x / cl;

    // settings of the row
    const float temperature = p.temperature ? p.temperature[r] : p.temperature_all;
    const int top_k = p.top_k ? p.top_k[r] : p.top_k_all;
    const float top_p = p.top_p ? p.top_p[r] : p.top_p_all;
    const float min_p = p.min_p ? p.min_p[r] : p.min_p_all;
    const bool greedy = !(temperature > 0.f);

    if (t < 64) {
        sh.tab.fix[t] = tabs.fix[t];
        sh.tab.flt[t] = tabs.flt[t];
    }

    // the warp's logits: into shared memory (cleaned), and the largest
    const long long first = (static_cast<long long>(rank) * SMP_WARPS + w) * chunk;
    const long long left = p.V - first;
    const int n = left <= 0 ? 0 : left < chunk ? static_cast<int>(left) : chunk;
    const T *row = static_cast<const T *>(p.Z) + r * p.ld + (n > 0 ? first : 0);
    const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    SmpChunk<T, SMEM> ck;
    ck.n = n;
    ck.aligned = aligned;
    float m = -INFINITY;
    if constexpr (SMEM) {
        T *mine = reinterpret_cast<T *>(smp_dyn) + static_cast<size_t>(w) * chunk;
        for (int i0 = l * 8; i0 < n; i0 += 4 * 256) {
            float x[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i0 + q * 256 < n) smp_load_global<T>(row + i0 + q * 256, n - i0 - q * 256, aligned, x[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i0 + q * 256 < n) {
                    smp_store_vec<T>(mine + i0 + q * 256, x[q]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = fmaxf(m, x[q][j]);
                }
        }
        ck.p = mine;
    } else {
        ck.p = row;
        for (int i = l * 8; i < n; i += 256) {
            float x[8];
            ck.load(i, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, x[j]);
        }
    }
    const int steps = (n + 255) / 256;   // sweeps of the warp over its logits

    int xs = 0;       // exchange slot in use
    // every CTA gives one value; afterwards sh.slot[xs ^ 1][k] holds that of rank k
    auto exchange = [&](uint32_t a, uint32_t b) {
        if (t < static_cast<int>(cl)) st_cluster_v4(map_to_rank(&sh.slot[xs][rank], t), a, b, 0u, 0u);
        cluster_sync_all();
        xs ^= 1;
    };

#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (l == 0) sh.red[w] = m;
    __syncthreads();
    m = sh.red[l & (SMP_WARPS - 1)];
#pragma unroll
    for (int o = SMP_WARPS / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // (the peers of the cluster have started: their shared memory may be written)
    cluster_sync_all();
    exchange(__float_as_uint(m), 0u);
    for (uint32_t k = 0; k < cl; ++k) m = fmaxf(m, __uint_as_float(sh.slot[xs ^ 1][k].x));

    if (m == -INFINITY || greedy) {
        // nothing to draw from, or the lowest index of the largest logit
        int best = 0x7fffffff;
        if (m != -INFINITY) {
            for (int s = 0; s < steps; ++s) {
                float x[8];
                ck.load(s * 256 + l * 8, x);
#pragma unroll
                for (int j = 7; j >= 0; --j)
                    if (x[j] == m && best > s * 256 + l * 8 + j) best = s * 256 + l * 8 + j;
            }
            best = __reduce_min_sync(0xffffffffu, best);
            if (best != 0x7fffffff) best += static_cast<int>(first);
            if (l == 0) sh.redlo[w] = static_cast<uint32_t>(best);
            __syncthreads();
            best = static_cast<int>(sh.redlo[l & (SMP_WARPS - 1)]);
            best = __reduce_min_sync(0xffffffffu, best);
            exchange(static_cast<uint32_t>(best), 0u);
            for (uint32_t k = 0; k < cl; ++k) best = min(best, static_cast<int>(sh.slot[xs ^ 1][k].x));
        }
        if (rank == 0 && t == 0) {
            p.tokens[r] = m == -INFINITY ? -1 : best;
            if (p.logprobs) p.logprobs[r] = m == -INFINITY ? -INFINITY : 0.f;
        }
        cluster_sync_all();   // no CTA leaves while a peer may still write into its slots
        return;
    }

    SmpRow rw;
    rw.m = m;
    rw.ih = 1.f / temperature;
    rw.il = fmaf(-temperature, rw.ih, 1.f) * rw.ih;
    if (!(fabsf(rw.il) < INFINITY)) rw.il = 0.f;   // temperatures near the ends of the type's range
    rw.c1 = tabs.c1;
    rw.c2 = tabs.c2;
    rw.c3 = tabs.c3;
    rw.inv = tabs.inv;

    const bool by_count = top_k > 0 && top_k < p.V;
    const bool by_weight = top_p < 1.f;
    // the cut: all logits with a key above cut_key are kept, and the first cut_ties of
    // those at it
    bool have_cut = false;
    uint32_t cut_key = 0, cut_ties = 0;

    if (by_count || by_weight) {
        int hb = 0;   // histogram in use
        // totals over the cluster of the histogram just filled; exclusive prefixes over
        // its bins into (pc, pw); then the bin in which `target` (a count, or a weight)
        // is reached
        auto totals = [&](uint32_t *pc, u64 *pw, uint32_t *tot_c, u64 *tot_w) {
            cluster_sync_all();
            uint32_t c = 0;
            u64 wt = 0;
            if (t < SMP_BINS) {
                for (uint32_t k = 0; k < cl; ++k) {
                    const uint4 h = ld_cluster_v4(map_to_rank(&sh.hist[hb][t], k));
                    c += h.x;
                    wt += static_cast<u64>(h.y) + (static_cast<u64>(h.z) << SMP_LIMB) +
                          (static_cast<u64>(h.w) << (2 * SMP_LIMB));
                }
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
        auto find = [&](const uint32_t *pc, const u64 *pw, uint32_t tot_c, u64 tot_w, bool count,
                        u64 target) {
            if (t < SMP_BINS) {
                const uint32_t c0 = pc[t], c1 = t + 1 < SMP_BINS ? pc[t + 1] : tot_c;
                const u64 w0 = pw[t], w1 = t + 1 < SMP_BINS ? pw[t + 1] : tot_w;
                const u64 a = count ? c0 : w0, b = count ? c1 : w1;
                if (a < target && target <= b) {
                    sh.bin = t;
                    sh.bc = c0;
                    sh.bcin = c1 - c0;
                    sh.bw = w0;
                    sh.bwin = w1 - w0;
                }
            }
            __syncthreads();
        };
        auto clear = [&]() {
            if (t < SMP_BINS) sh.hist[hb][t] = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
        };

        // first level: x in steps of 1/8
        clear();
        for (int s = 0; s < steps; ++s) {
            float x[8];
            ck.load(s * 256 + l * 8, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xx = smp_x(x[j], rw);
                const int b = xx < SMP_X_END ? static_cast<int>(xx * SMP_BINS_PER_UNIT) : -1;
                if (by_weight) smp_hist_add<true>(sh.hist[hb], b, smp_weight(x[j], rw, sh.tab), l);
                else smp_hist_add<false>(sh.hist[hb], b, 0ull, l);
            }
        }
        uint32_t tot_c;
        u64 tot_w;
        totals(sh.l0c, sh.l0w, &tot_c, &tot_w);

        // the key and the number of equal logits at which `target` is reached
        auto search = [&](bool count, u64 target, uint32_t *key, uint32_t *ties, u64 *kept_w) {
            find(sh.l0c, sh.l0w, tot_c, tot_w, count, target);
            const int b0 = sh.bin;
            uint32_t base_c = sh.bc;
            u64 base_w = sh.bw;
            // the keys in that bin
            uint32_t klo = 0xffffffffu, khi = 0u;
            for (int s = 0; s < steps; ++s) {
                float x[8];
                ck.load(s * 256 + l * 8, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xx = smp_x(x[j], rw);
                    if (xx < SMP_X_END && static_cast<int>(xx * SMP_BINS_PER_UNIT) == b0) {
                        const uint32_t k = smp_key<T>(x[j]);
                        klo = min(klo, k);
                        khi = max(khi, k);
                    }
                }
            }
            klo = __reduce_min_sync(0xffffffffu, klo);
            khi = __reduce_max_sync(0xffffffffu, khi);
            if (l == 0) {
                sh.redlo[w] = klo;
                sh.redhi[w] = khi;
            }
            __syncthreads();
            klo = __reduce_min_sync(0xffffffffu, sh.redlo[l & (SMP_WARPS - 1)]);
            khi = __reduce_max_sync(0xffffffffu, sh.redhi[l & (SMP_WARPS - 1)]);
            exchange(klo, khi);
            for (uint32_t k = 0; k < cl; ++k) {
                klo = min(klo, sh.slot[xs ^ 1][k].x);
                khi = max(khi, sh.slot[xs ^ 1][k].y);
            }
            while (true) {
                const int bits = 32 - __clz(khi - klo);
                const int shift = bits > 8 ? bits - 8 : 0;
                clear();
                for (int s = 0; s < steps; ++s) {
                    float x[8];
                    ck.load(s * 256 + l * 8, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t k = smp_key<T>(x[j]);
                        const int b = k >= klo && k <= khi ? static_cast<int>((khi - k) >> shift) : -1;
                        if (by_weight)
                            smp_hist_add<true>(sh.hist[hb], b, b >= 0 ? smp_weight(x[j], rw, sh.tab) : 0ull, l);
                        else
                            smp_hist_add<false>(sh.hist[hb], b, 0ull, l);
                    }
                }
                uint32_t tc;
                u64 tw;
                totals(sh.rc, sh.rw, &tc, &tw);
                find(sh.rc, sh.rw, tc, tw, count, target - (count ? static_cast<u64>(base_c) : base_w));
                const uint32_t b = static_cast<uint32_t>(sh.bin);
                base_c += sh.bc;
                base_w += sh.bw;
                if (shift == 0) {
                    *key = khi - b;
                    const u64 one = sh.bwin / sh.bcin;   // equal logits, equal weights
                    *ties = count ? static_cast<uint32_t>(target) - base_c
                                  : static_cast<uint32_t>((target - base_w + one - 1) / one);
                    *kept_w = base_w + static_cast<u64>(*ties) * one;
                    __syncthreads();
                    return;
                }
                const uint32_t hi = khi - (b << shift);
                const uint32_t width = (1u << shift) - 1u;
                klo = hi - klo > width ? hi - width : klo;
                khi = hi;
                __syncthreads();
            }
        };

        u64 pool = tot_w;   // weight of what top-k keeps
        if (by_count && static_cast<uint32_t>(top_k) < tot_c) {
            search(true, static_cast<u64>(top_k), &cut_key, &cut_ties, &pool);
            have_cut = true;
        }
        if (by_weight) {
            u64 target = top_p > 0.f ? smp_mul_floor(top_p, pool, true) : 1ull;
            if (target == 0) target = 1;
            uint32_t key, ties;
            u64 kept;
            search(false, target, &key, &ties, &kept);
            if (!have_cut || key > cut_key || (key == cut_key && ties < cut_ties)) {
                cut_key = key;
                cut_ties = ties;
            }
            have_cut = true;
        }
    }

    // kept: weight at least w_min, and the cut
    u64 w_min = 0;
    if (min_p > 0.f)
        w_min = min_p >= 1.f ? 1ull << SMP_ONE_SHIFT : smp_mul_floor(min_p, 1ull << SMP_ONE_SHIFT, true);
    const u64 tie_w0 = have_cut ? smp_weight(smp_unkey<T>(cut_key), rw, sh.tab) : 0ull;
    const u64 tie_w = tie_w0 >= w_min ? tie_w0 : 0ull;
    // weight above the cut (tie: at the cut) of one logit
    auto kept_weight = [&](float x, bool *tie) -> u64 {
        *tie = false;
        if (have_cut) {
            const uint32_t k = smp_key<T>(x);
            if (k < cut_key) return 0ull;
            if (k == cut_key) {
                *tie = true;
                return 0ull;
            }
        }
        const u64 v = smp_weight(x, rw, sh.tab);
        return v >= w_min ? v : 0ull;
    };

    // sums of every warp of the cluster, in index order
    u64 above = 0;
    uint32_t ties = 0;
    for (int s = 0; s < steps; ++s) {
        float x[8];
        ck.load(s * 256 + l * 8, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bool tie;
            above += kept_weight(x[j], &tie);
            ties += tie ? 1u : 0u;
        }
    }
    above = warp_sum64(above);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (l < static_cast<int>(cl))
        st_cluster_v4(map_to_rank(&sh.wslot[rank * SMP_WARPS + w], l), static_cast<uint32_t>(above),
                      static_cast<uint32_t>(above >> 32), ties, 0u);
    cluster_sync_all();

    // every warp sums all warps' entries: 4 per lane, in order
    constexpr int PER_LANE = SMP_MAX_CLUSTER * SMP_WARPS / 32;
    const int entries = static_cast<int>(cl) * SMP_WARPS;
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
    const int me = static_cast<int>(rank) * SMP_WARPS + w;
    u64 lane_w = 0, my_before = 0;
    uint32_t my_ties_before = 0;
#pragma unroll
    for (int q = 0; q < PER_LANE; ++q) {
        if (l * PER_LANE + q == me) {
            my_before = lane_w;
            my_ties_before = before_t;
        }
        const uint32_t room = before_t < cut_ties ? cut_ties - before_t : 0u;
        lane_w += ew[q] + static_cast<u64>(et[q] < room ? et[q] : room) * tie_w;
        before_t += et[q];
    }
    u64 incl = lane_w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = shfl_up64(incl, o);
        if (l >= o) incl += v;
    }
    const u64 total = __shfl_sync(0xffffffffu, incl, 31);
    const int owner = me / PER_LANE;
    const u64 my_first = __shfl_sync(0xffffffffu, my_before + incl - lane_w, owner);
    my_ties_before = __shfl_sync(0xffffffffu, my_ties_before, owner);
    const uint32_t my_room = my_ties_before < cut_ties ? cut_ties - my_ties_before : 0u;
    const u64 my_sum = above + static_cast<u64>(ties < my_room ? ties : my_room) * tie_w;

    // the first index whose cumulative weight exceeds u * total
    const float u = p.u[r];
    u64 target = total - 1;
    if (u < 1.f) target = u > 0.f ? smp_mul_floor(u, total, false) : 0ull;
    if (target >= my_first && target - my_first < my_sum) {
        u64 run = my_first;
        uint32_t seen = my_ties_before;
        for (int s = 0; s < steps; ++s) {
            const int i = s * 256 + l * 8;
            float x[8];
            u64 v[8];
            uint32_t tmask = 0;
            ck.load(i, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bool tie;
                v[j] = kept_weight(x[j], &tie);
                if (tie) tmask |= 1u << j;
            }
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
            if (hit) {
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
                    p.tokens[r] = first + i + at;
                    if (p.logprobs) {
                        constexpr float UNIT = 1.f / static_cast<float>(1ull << SMP_ONE_SHIFT);
                        const u64 one = 1ull << SMP_ONE_SHIFT;
                        // log(total): the largest logit's weight is 1, so near 0 by log1p
                        const float ls = total < 2 * one ? log1pf(static_cast<float>(total - one) * UNIT)
                                                         : logf(static_cast<float>(total) * UNIT);
                        p.logprobs[r] = -smp_x(z, rw) - ls;
                    }
                }
                break;
            }
            run += __shfl_sync(0xffffffffu, in, 31);
            seen += __shfl_sync(0xffffffffu, tb, 31);
        }
    }
    cluster_sync_all();   // no CTA leaves while a peer may still use its shared memory
}

using SampleKernel = void (*)(const SampleParams, const SampleTables, const int);

SampleKernel sample_kernel(int dtype, bool smem) {
    if (dtype == CE_FP32) return smem ? lce_sample_kernel<float, true> : lce_sample_kernel<float, false>;
    if (dtype == CE_FP16) return smem ? lce_sample_kernel<__half, true> : lce_sample_kernel<__half, false>;
    return smem ? lce_sample_kernel<__nv_bfloat16, true> : lce_sample_kernel<__nv_bfloat16, false>;
}

constexpr int SMP_MAX_DYN = 160 * 1024;   // a CTA's logits; the rest of its shared memory is static

}  // namespace

cudaError_t sample_set_attributes() {
    for (int dt = CE_BF16; dt <= CE_FP16; ++dt) {
        const cudaError_t e = cudaFuncSetAttribute(
            sample_kernel(dt, true), cudaFuncAttributeMaxDynamicSharedMemorySize, SMP_MAX_DYN);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_sample(const SampleParams &p, cudaStream_t s) {
    if (p.N <= 0) return cudaSuccess;
    static const SampleTables tabs = make_sample_tables();
    const long long elem = p.dtype == CE_FP32 ? 4 : 2;
    int cl = 1;
    long long chunk = 0;
    for (;; cl *= 2) {
        chunk = (p.V + cl * SMP_WARPS - 1) / (cl * SMP_WARPS);
        chunk = (chunk + 7) / 8 * 8;
        if (cl == SMP_MAX_CLUSTER || chunk <= 256) break;
    }
    const long long bytes = chunk * SMP_WARPS * elem;
    const bool smem = bytes <= SMP_MAX_DYN;
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
    return cudaLaunchKernelEx(&cfg, sample_kernel(p.dtype, smem), p, tabs, static_cast<int>(chunk));
}

}  // namespace lce
