// Losses on answers: what the log probabilities of drawn tokens are worth, and the gradient.
//
//   * rows of given logits: log p of the row's label, the clipped policy loss with its KL term
//     and the gradient (p - onehot) * scale in one pass over the logits (cluster kernel), or
//     in two for rows beyond eight CTAs' shared memory (streaming kernel);
//   * pairs: log probabilities added up over each sequence, the loss of the paired log ratios,
//     and the coefficient that each row's p - onehot gets;
//   * the gradient of a preference over given logits, once those coefficients are known.
//
// Rows may start anywhere (an odd vocabulary in dense rows): a row is a head of fewer than 16
// bytes, whole 16-byte vectors, and a tail; no byte beside it is read or written. Rows that do
// not count are not read; their gradient is zeros. Every sum has a fixed order.
#include <map>
#include <mutex>
#include <type_traits>

#include <cuda_fp16.h>

#include "lce_internal.h"
#include "lce_ptx.cuh"

namespace lce {

namespace {

constexpr int ANS_THREADS = 512;
constexpr int ANS_WARPS = ANS_THREADS / 32;
constexpr int ANS_MAX_CLUSTER = 8;
constexpr int ANS_MAX_BUF = 3;
constexpr int ANS_SLOTS = 4;                     // rows between their sums and their results
constexpr uint32_t ANS_COPY_BYTES = 32768;       // bytes per bulk copy instruction
constexpr uint64_t ANS_WAIT_NS = 2000000000ull;  // bound of every wait (2 s)
constexpr int STREAM_THREADS = 1024;
constexpr long long SCAN_ONE_CTA = 32768;        // labels that one CTA scans

// A 16-byte vector of logits seen as fp32 pairs.
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int ELEMS = 8, PAIRS = 4;
    static constexpr uint32_t NEG_INF = 0xff80ff80u;
    __device__ static float2 pair(const uint4 &u, int q) {
        const uint32_t w = (&u.x)[q];
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ static void set_pair(uint4 &u, int q, float2 v) { (&u.x)[q] = pack_bf16x2(v.x, v.y); }
    // The largest of N vectors' values and m.
    template <int N> __device__ static float max_of(const uint4 (&u)[N], float m) {
        __nv_bfloat162 a = reinterpret_cast<const __nv_bfloat162 *>(&u[0])[0];
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) a = __hmax2(a, reinterpret_cast<const __nv_bfloat162 *>(&u[i / 4])[i % 4]);
        return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
    }
    __device__ static __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Vec<__half> {
    static constexpr int ELEMS = 8, PAIRS = 4;
    static constexpr uint32_t NEG_INF = 0xfc00fc00u;
    __device__ static float2 pair(const uint4 &u, int q) {
        return __half22float2(reinterpret_cast<const __half2 *>(&u)[q]);
    }
    __device__ static void set_pair(uint4 &u, int q, float2 v) { (&u.x)[q] = pack_f16x2(v.x, v.y); }
    template <int N> __device__ static float max_of(const uint4 (&u)[N], float m) {
        __half2 a = reinterpret_cast<const __half2 *>(&u[0])[0];
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) a = __hmax2(a, reinterpret_cast<const __half2 *>(&u[i / 4])[i % 4]);
        return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
    }
    __device__ static __half from(float v) { return __float2half_rn(v); }
};
template <> struct Vec<float> {
    static constexpr int ELEMS = 4, PAIRS = 2;
    static constexpr uint32_t NEG_INF = 0xff800000u;
    __device__ static float2 pair(const uint4 &u, int q) {
        return make_float2(__uint_as_float((&u.x)[2 * q]), __uint_as_float((&u.x)[2 * q + 1]));
    }
    __device__ static void set_pair(uint4 &u, int q, float2 v) {
        (&u.x)[2 * q] = __float_as_uint(v.x);
        (&u.x)[2 * q + 1] = __float_as_uint(v.y);
    }
    template <int N> __device__ static float max_of(const uint4 (&u)[N], float m) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(u[i].x), __uint_as_float(u[i].y))),
                      fmaxf(__uint_as_float(u[i].z), __uint_as_float(u[i].w)));
        return m;
    }
    __device__ static float from(float v) { return v; }
};

__device__ __forceinline__ float wmax(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float wsum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Over groups of G consecutive lanes.
template <int G> __device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int G> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// A sum kept as two fp32 numbers (what the first addition loses goes into the second): losses of
// either sign add up to far less than they are, and fp64 runs at a sixty-fourth of the rate.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ void add(float v) {
        const float s = hi + v, b = s - hi;
        lo += (hi - (s - b)) + (v - b);
        hi = s;
    }
    __device__ void warp() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
            // (the larger first, so that both lanes of a pair get the same bits)
            const float s = hi + h, b = s - hi, c = s - h;
            lo = (lo + l) + (fabsf(hi) >= fabsf(h) ? (h - b) : (hi - c));
            hi = s;
        }
    }
    // An infinity or a NaN leaves a NaN in `lo`: the sum is then `hi` alone.
    __device__ double value() const { return lo == lo ? static_cast<double>(hi) + lo : static_cast<double>(hi); }
};
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t cluster_id() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_count() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Stores four words into the shared memory of a CTA of the cluster, completing 16 bytes of
// transaction on its mbarrier `bar`.
__device__ __forceinline__ void st_async_f32x4(uint32_t addr, float a, float b, float c, float d,
                                               uint32_t bar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
        "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void wait_for_previous_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// A row of V values as a head of `head` values, `nvec` vectors and a tail.
template <typename T> struct RowSplit {
    const T *row;
    int head;
    long long nvec, tail0;
    __device__ RowSplit(const T *r, long long V) : row(r) {
        constexpr int EL = Vec<T>::ELEMS;
        const int off = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
        head = off ? EL - off : 0;
        if (head > V) head = static_cast<int>(V);
        nvec = (V - head) / EL;
        tail0 = head + nvec * EL;
    }
    // The value beside the vectors that thread t holds (head first, then tail), or -1.
    __device__ long long scalar(int t, long long V) const {
        const long long i = t < head ? t : tail0 + (t - head);
        return i < V ? i : -1;
    }
};

// exp((z - m) / T) as 2^(z k2 + nm) * c for k2 = log2(e) / T: one fused operation for each logit. nm is
// -m k2 as fp32 has it and c takes back what that rounding lost, so the result is as exact as
// the distance from m is. That loss is up to half a unit of nm: an eighth below 2^22, but beyond what a power of two
// can hold (c 0, the other factor infinite) for masks of -1e10 or a temperature of 1e-9. From 2^22 on `far` is
// set, and the distance is formed first: one operation more.
constexpr float EXP_FUSED_BELOW = 0x1p22f;
struct ExpFrom {
    float m, k2, nm, c;
    bool far;
    __device__ ExpFrom(float m_, float k2_) : m(m_ == -INFINITY ? 0.f : m_), k2(k2_) {
        nm = -(m * k2);
        far = !(fabsf(nm) < EXP_FUSED_BELOW);
        c = far ? 1.f : exp2_fast(-fmaf(m, k2, nm));
        if (far) nm = 0.f;
    }
    __device__ float operator()(float z) const { return exp2_fast(far ? (z - m) * k2 : fmaf(z, k2, nm)); }
    __device__ float2 pair(float2 z) const {
        const float2 a = __ffma2_rn(z, make_float2(k2, k2), make_float2(nm, nm));
        return make_float2(exp2_fast(a.x), exp2_fast(a.y));
    }
    __device__ float2 far_pair(float2 z) const {
        const float2 a = __fmul2_rn(__fadd2_rn(z, make_float2(-m, -m)), make_float2(k2, k2));
        return make_float2(exp2_fast(a.x), exp2_fast(a.y));
    }
};

__device__ __forceinline__ bool label_counts(long long v, long long V, long long ign) {
    return v != ign && v >= 0 && v < V;
}

// Whether this CTA is the last of `total` to come here; all that they wrote before is visible to it.
__device__ __forceinline__ bool last_to_finish(int *done, int total, int *s_last) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        *s_last = atomicAdd(done, 1) == total - 1;
        __threadfence();
    }
    __syncthreads();
    return *s_last != 0;
}

// The sum of v[0 .. n) in a fixed order, by all threads of a CTA (in thread 0).
__device__ __forceinline__ double block_sum(const float *v, long long n, float2 *s_red) {
    const int t = threadIdx.x, nt = blockDim.x;
    Sum2 s;
#pragma unroll 4
    for (long long i = t; i < n; i += nt) s.add(__ldcg(v + i));
    s.warp();
    if ((t & 31) == 0) s_red[t >> 5] = make_float2(s.hi, s.lo);
    __syncthreads();
    if (t < 32) {
        const float2 x = t < nt / 32 ? s_red[t] : make_float2(0.f, 0.f);
        s.hi = x.x;
        s.lo = x.y;
        s.warp();
    }
    __syncthreads();
    return s.value();
}

__device__ __forceinline__ void write_loss(const AnswerParams &p, float2 *s_red) {
    const double s = block_sum(p.loss_rows, p.N, s_red);
    if (threadIdx.x == 0) {
        const int nv = p.hdr[HDR_NVALID];
        *p.loss = !p.mean ? static_cast<float>(s) : nv > 0 ? static_cast<float>(s / nv) : 0.f;
    }
}

// ------------------------------------------------------------------ labels

// One CTA: the counting rows and the range check, written (not added) into the header.
__global__ void __launch_bounds__(1024) lce_answer_scan_kernel(const long long *__restrict__ y, long long N,
                                                               long long V, long long ign, int *hdr) {
    __shared__ int s_cnt[32], s_bad[32];
    let_next_grid_start();
    int cnt = 0, bad = 0;
#pragma unroll 4
    for (long long i = threadIdx.x; i < N; i += 1024) {
        const long long v = y[i];
        const bool ok = label_counts(v, V, ign);
        cnt += ok;
        bad |= !ok && v != ign;
    }
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    bad = __reduce_or_sync(0xffffffffu, bad);
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    if (l == 0) {
        s_cnt[w] = cnt;
        s_bad[w] = bad;
    }
    __syncthreads();
    if (w == 0) {
        cnt = __reduce_add_sync(0xffffffffu, s_cnt[l]);
        bad = __reduce_or_sync(0xffffffffu, s_bad[l]);
        if (l < HDR_COUNTERS) hdr[l] = l == HDR_FLAG ? (bad ? FLAG_LABEL : 0) : l == HDR_NVALID ? cnt : 0;
    }
}

// ------------------------------------------------------------------ rows, cluster kernel
// A cluster of 1, 2, 4 or 8 CTAs takes one row at a time; rank k owns the vectors [k sv, (k + 1) sv)
// of it, rank 0 also the values beside them. The logits stay in shared memory from the copy that
// brings them to the gradient: nbuf buffers hold a row that comes, one that is summed and one
// whose gradient is written. Rows that count go through three stages:
//   * a producer warp starts the bulk copies of a row as soon as a buffer is free;
//   * 16 warps sum row i: per thread the maximum and the sum of exp((z - maximum) / T), merged over
//     the warp and left for the manager; then they write the gradient of row i - 1,
//     exp((z - max) / T) * (scale / sum), the label's less `scale`. (The exponentials are formed twice:
//     kept in 16 bits they would be rounded.)
//   * a manager warp merges the warps' parts, exchanges (max, sum, the label's logit) with the cluster's
//     other CTAs by st.async, and forms the log probability, the row's loss and the gradient's
//     scale once, while the 16 warps are at another row.
// Every sum has a fixed order. Rows that do not count take no buffer: their zeros are written on the way.

struct RowResult {
    float M, f, scale, zl;   // maximum, scale / sum, scale, the label's logit
};

template <typename T>
__global__ void __launch_bounds__(ANS_THREADS + 64, 1)
    lce_answer_rows_kernel(const __grid_constant__ AnswerParams p, const int sv, const int nbuf) {
    using CV = Vec<T>;
    constexpr int EL = CV::ELEMS;
    extern __shared__ __align__(128) uint8_t ans_smem[];
    __shared__ __align__(8) uint64_t lbar[ANS_MAX_BUF];    // a row's copies landed
    __shared__ __align__(8) uint64_t ebar[ANS_MAX_BUF];    // every warp, the manager too, is done with the buffer
    __shared__ __align__(8) uint64_t sbar[ANS_SLOTS];      // every warp's part of the row is there
    __shared__ __align__(8) uint64_t xbar[ANS_SLOTS];      // every CTA's part of the row landed
    __shared__ __align__(8) uint64_t rbar[ANS_SLOTS];      // the row's result is there
    __shared__ __align__(16) float4 xslot[ANS_SLOTS][ANS_MAX_CLUSTER];
    __shared__ __align__(16) RowResult s_res[ANS_SLOTS];
    __shared__ float2 s_part[ANS_SLOTS][ANS_WARPS];
    __shared__ float2 s_red[ANS_WARPS + 2];
    __shared__ int s_abort, s_last;

    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    const uint32_t rank = cluster_ctarank(), cl = cluster_ctas();
    const long long cid = cluster_id(), ncl = cluster_count();
    const Abort ab{&s_abort, p.hdr, ANS_WAIT_NS};
    const T *Z = static_cast<const T *>(p.Z);
    const float k2 = LOG2E_F * p.pol.inv_t;

    if (t == 0) {
        s_abort = 0;
        for (int b = 0; b < nbuf; ++b) {
            mbar_init(&lbar[b], 1);
            mbar_init(&ebar[b], ANS_WARPS + 1);
        }
        for (int b = 0; b < ANS_SLOTS; ++b) {
            mbar_init(&sbar[b], ANS_WARPS);
            mbar_init(&xbar[b], 1);
            mbar_init(&rbar[b], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    cluster_sync_all();   // every CTA's barriers exist before a peer signals them

    const long long v0 = static_cast<long long>(rank) * sv;
    // vectors of a row that this CTA owns
    auto vectors = [&](const RowSplit<T> &rs) -> int {
        const long long n = rs.nvec - v0;
        return n <= 0 ? 0 : n < sv ? static_cast<int>(n) : sv;
    };
    auto label = [&](long long r) -> long long { return r < p.N ? p.y[r] : p.ignore_index; };
    auto counts = [&](long long yv) -> bool { return label_counts(yv, p.V, p.ignore_index); };
    auto buffer = [&](int b) -> uint8_t * { return ans_smem + static_cast<size_t>(b) * sv * 16; };
    // (a wait that runs out ends the loop for a whole warp: its lanes decide together)

    if (w == ANS_WARPS) {
        // the producer
        if (l == 0) {
            int b = 0;
            uint32_t par = 1;   // (the buffers are free at first)
            long long issued = 0, y_next = label(cid);
            for (long long r = cid; r < p.N; r += ncl) {
                const long long yv = y_next;
                y_next = label(r + ncl);
                if (!counts(yv)) continue;
                if (!mbar_wait(&ebar[b], par, ab)) break;
                const RowSplit<T> rs(Z + r * p.ld, p.V);
                const uint32_t bytes = vectors(rs) * 16u;
                ++issued;
                if (bytes == 0) {
                    mbar_arrive(&lbar[b]);
                } else {
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(&lbar[b], bytes);
                    const uint8_t *src = reinterpret_cast<const uint8_t *>(rs.row + rs.head + v0 * EL);
                    const uint32_t dst = smem_u32(buffer(b));
                    for (uint32_t off = 0; off < bytes; off += ANS_COPY_BYTES)
                        bulk_copy(dst + off, src + off, bytes - off < ANS_COPY_BYTES ? bytes - off : ANS_COPY_BYTES,
                                  smem_u32(&lbar[b]));
                }
                if (++b == nbuf) {
                    b = 0;
                    par ^= 1u;
                }
            }
            // copies that nobody waited for (after a wait that ran out) may still be landing
            for (long long j = issued > nbuf ? issued - nbuf : 0; j < issued; ++j)
                mbar_wait_drain(&lbar[j % nbuf], static_cast<uint32_t>((j / nbuf) & 1), ANS_WAIT_NS);
        }
    } else if (w == ANS_WARPS + 1) {
        // the manager
        int b = 0, xs = 0;
        uint32_t lpar = 0, xpar = 0;
        long long y_next = label(cid);
        wait_for_previous_grid();   // the header
        const int nvalid = p.hdr[HDR_NVALID];
        for (long long r = cid; r < p.N; r += ncl) {
            const long long yv = y_next;
            y_next = label(r + ncl);
            if (!counts(yv)) {
                if (l == 0 && rank == 0) {
                    p.loss_rows[r] = 0.f;
                    if (p.pol.logp) p.pol.logp[r] = 0.f;
                    if (p.max_sum) p.max_sum[r] = make_float2(0.f, 1.f);
                }
                continue;
            }
            const RowSplit<T> rs(Z + r * p.ld, p.V);
            if (!__all_sync(0xffffffffu, mbar_wait(&lbar[b], lpar, ab))) break;
            // the label's logit, if it lies here
            float zl = 0.f;
            if (yv >= rs.head && yv < rs.tail0) {
                const long long yi = yv - rs.head - v0 * EL;
                if (yi >= 0 && yi < static_cast<long long>(vectors(rs)) * EL)
                    zl = static_cast<float>(reinterpret_cast<const T *>(buffer(b))[yi]);
            } else if (rank == 0) {
                zl = static_cast<float>(rs.row[yv]);
            }
            __syncwarp();
            if (l == 0) {
                mbar_arrive(&ebar[b]);
                mbar_arrive_expect_tx(&xbar[xs], cl * 16u);
            }
            const PolicyInputs in = lce_policy_inputs(p.pol, r);
            const float d = lce_row_scale(p.dloss, p.dloss_per_row, p.mean, nvalid, r, true);
            if (!__all_sync(0xffffffffu, mbar_wait(&sbar[xs], xpar, ab))) break;
            const float2 x = s_part[xs][l % ANS_WARPS];
            float M = group_max<ANS_WARPS>(x.x);
            float S = group_sum<ANS_WARPS>(x.x == -INFINITY ? x.y : x.y * exp2_fast((x.x - M) * k2));   // (0, or a NaN, without a logit)
            if (l < static_cast<int>(cl))
                st_async_f32x4(map_to_rank(&xslot[xs][rank], l), M, S, zl, 0.f, map_to_rank(&xbar[xs], l));
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(&xbar[xs], xpar, ab))) break;
            const int part = l % ANS_MAX_CLUSTER;
            const float4 q = part < static_cast<int>(cl) ? xslot[xs][part] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            M = group_max<ANS_MAX_CLUSTER>(q.x);
            S = group_sum<ANS_MAX_CLUSTER>(q.x == -INFINITY ? q.y : q.y * exp2_fast((q.x - M) * k2));
            zl = group_sum<ANS_MAX_CLUSTER>(q.z);
            const float logp = (zl - M) * p.pol.inv_t - logf(S);
            PolicyRow pr{-logp, 0.f};
            if (p.pol.adv) pr = lce_policy_row(p.pol, in, logp);
            if (l == 0) {
                const float scale = -pr.slope * p.pol.inv_t * d;
                s_res[xs] = RowResult{M, scale / S, scale, zl};
                mbar_arrive(&rbar[xs]);
                if (rank == 0) {
                    p.loss_rows[r] = pr.loss;
                    if (p.pol.logp) p.pol.logp[r] = logp;
                    if (p.max_sum) p.max_sum[r] = make_float2(M, S);
                }
            }
            __syncwarp();
            if (++b == nbuf) {
                b = 0;
                lpar ^= 1u;
            }
            if (++xs == ANS_SLOTS) {
                xs = 0;
                xpar ^= 1u;
            }
        }
    } else {
        // the row before, whose gradient is to be written (prev < 0: none), and its buffer
        long long prev = -1, prev_y = 0;
        int b = 0, xs = 0, prev_b = 0, prev_xs = 0;
        uint32_t lpar = 0, xpar = 0, prev_par = 0;
        auto zeros = [&](long long r, const RowSplit<T> &rs) {
            if (!p.dZ) return;
            T *drow = static_cast<T *>(p.dZ) + r * p.ld;
            uint4 *dvec = reinterpret_cast<uint4 *>(drow + rs.head) + v0;
            const int n = vectors(rs);
            for (int v = t; v < n; v += ANS_THREADS) dvec[v] = make_uint4(0u, 0u, 0u, 0u);
            const long long si = rank == 0 && w == 0 ? rs.scalar(t, p.V) : -1;
            if (si >= 0) drow[si] = CV::from(0.f);
        };
        // The gradient of the row before; its buffer is free after that.
        auto gradient = [&]() -> bool {
            if (prev < 0) return true;
            if (!__all_sync(0xffffffffu, mbar_wait(&rbar[prev_xs], prev_par, ab))) return false;
            if (p.dZ) {
                const RowResult res = s_res[prev_xs];
                const RowSplit<T> rs(Z + prev * p.ld, p.V);
                if (res.scale == 0.f) {
                    zeros(prev, rs);
                } else {
                    T *drow = static_cast<T *>(p.dZ) + prev * p.ld;
                    uint4 *dvec = reinterpret_cast<uint4 *>(drow + rs.head) + v0;
                    const uint4 *sg = reinterpret_cast<const uint4 *>(buffer(prev_b));
                    const int n = vectors(rs);
                    const ExpFrom e(res.M, k2);
                    const float f = res.f * e.c;
                    const float2 f2 = make_float2(f, f);
                    auto one = [&](const uint4 &u, auto far) {
                        uint4 out;
#pragma unroll
                        for (int q = 0; q < CV::PAIRS; ++q) {
                            const float2 z = CV::pair(u, q);
                            CV::set_pair(out, q, __fmul2_rn(decltype(far)::value ? e.far_pair(z) : e.pair(z), f2));
                        }
                        return out;
                    };
                    if (!e.far) {
#pragma unroll 1
                        for (int v = t; v < n; v += 2 * ANS_THREADS) {
                            const bool two = v + ANS_THREADS < n;
                            const uint4 u0 = sg[v], u1 = two ? sg[v + ANS_THREADS] : u0;
                            dvec[v] = one(u0, std::false_type());
                            if (two) dvec[v + ANS_THREADS] = one(u1, std::false_type());
                        }
                    } else {
#pragma unroll 1
                        for (int v = t; v < n; v += ANS_THREADS) dvec[v] = one(sg[v], std::true_type());
                    }
                    const long long si = rank == 0 && w == 0 ? rs.scalar(t, p.V) : -1;
                    if (si >= 0) drow[si] = CV::from(e(static_cast<float>(rs.row[si])) * f);
                    // the label's place again, by the thread that has written it
                    const long long yi = prev_y - rs.head - v0 * EL;
                    const bool mine = prev_y >= rs.head && prev_y < rs.tail0
                                          ? yi >= 0 && yi < static_cast<long long>(n) * EL &&
                                                static_cast<int>(yi / EL) % ANS_THREADS == t
                                          : si == prev_y;
                    if (mine) drow[prev_y] = CV::from(e(res.zl) * f - res.scale);
                }
            }
            __syncwarp();
            if (l == 0) mbar_arrive(&ebar[prev_b]);
            prev = -1;
            return true;
        };
        long long y_next = label(cid), used = 0;
        bool ok = true;
        for (long long r = cid; r < p.N; r += ncl) {
            const long long yv = y_next;
            y_next = label(r + ncl);
            const RowSplit<T> rs(Z + r * p.ld, p.V);
            if (!counts(yv)) {
                zeros(r, rs);
                continue;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&lbar[b], lpar, ab));
            if (!ok) break;
            // this row's maximum and sum, four vectors of each thread at a time
            const uint4 *sg = reinterpret_cast<const uint4 *>(buffer(b));
            const int n = vectors(rs);
            const long long si = rank == 0 && w == 0 ? rs.scalar(t, p.V) : -1;
            float m = si >= 0 ? static_cast<float>(rs.row[si]) : -INFINITY;
            float s = si >= 0 ? (m == -INFINITY ? 0.f : m == m ? 1.f : m) : 0.f;
            if (m != m) m = -INFINITY;
#pragma unroll 1
            for (int v = t; v < n; v += 4 * ANS_THREADS) {
                uint4 u[4];
                if (v + 3 * ANS_THREADS < n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[j] = sg[v + j * ANS_THREADS];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        u[j] = v + j * ANS_THREADS < n
                                   ? sg[v + j * ANS_THREADS]
                                   : make_uint4(CV::NEG_INF, CV::NEG_INF, CV::NEG_INF, CV::NEG_INF);
                }
                const float mv = CV::max_of(u, m);
                const ExpFrom e(mv, k2);
                float2 a0 = make_float2(0.f, 0.f), a1 = make_float2(0.f, 0.f);
                if (!e.far) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int q = 0; q < CV::PAIRS; ++q) {
                            if (q & 1) a1 = __fadd2_rn(a1, e.pair(CV::pair(u[j], q)));
                            else a0 = __fadd2_rn(a0, e.pair(CV::pair(u[j], q)));
                        }
                    a0 = __fadd2_rn(a0, a1);
                } else {
#pragma unroll 1
                    for (int i = v; i < n && i < v + 4 * ANS_THREADS; i += ANS_THREADS) {
                        const uint4 w4 = sg[i];
#pragma unroll
                        for (int q = 0; q < CV::PAIRS; ++q) a0 = __fadd2_rn(a0, e.far_pair(CV::pair(w4, q)));
                    }
                }
                // (without a logit so far every exponential is 0, or a NaN)
                s = s * (m == mv ? 1.f : exp2_fast((m - mv) * k2)) + (a0.x + a0.y) * e.c;
                m = mv;
            }
            const float wm = wmax(m);
            const float ws = wsum(m == -INFINITY ? s : s * exp2_fast((m - wm) * k2));   // (0, or a NaN, without a logit)
            // (the slot is free: with a gradient every warp has waited for the row before; without
            // one the row that had it last is waited for here)
            if (!p.dZ && used >= ANS_SLOTS) {
                ok = __all_sync(0xffffffffu, mbar_wait(&rbar[xs], xpar ^ 1u, ab));
                if (!ok) break;
            }
            ++used;
            if (l == 0) {
                s_part[xs][w] = make_float2(wm, ws);
                mbar_arrive(&sbar[xs]);
                if (!p.dZ) mbar_arrive(&ebar[b]);   // (no gradient will read it again)
            }
            __syncwarp();
            if (p.dZ) {
                ok = gradient();
                if (!ok) break;
                prev = r;
                prev_y = yv;
                prev_b = b;
                prev_xs = xs;
                prev_par = xpar;
            }
            if (++b == nbuf) {
                b = 0;
                lpar ^= 1u;
            }
            if (++xs == ANS_SLOTS) {
                xs = 0;
                xpar ^= 1u;
            }
        }
        if (ok) gradient();
    }
    __syncthreads();
    cluster_sync_all();   // no CTA leaves while a peer may still write into its slots
    if (rank == 0 && p.loss && last_to_finish(p.hdr + HDR_DONE, static_cast<int>(ncl), &s_last))
        write_loss(p, s_red);
}

// ------------------------------------------------------------------ rows, streaming kernel
// One CTA per row, two passes (a running max and sum, then the gradient), any V.

__device__ __forceinline__ void merge(float &m, float &s, float m2, float s2, float k2) {
    const float M = fmaxf(m, m2);
    if (M == -INFINITY) {
        s += s2;   // (0, or a NaN)
        return;
    }
    s = (m == -INFINITY ? s : s * exp2f((m - M) * k2)) + (m2 == -INFINITY ? s2 : s2 * exp2f((m2 - M) * k2));
    m = M;
}

// Row r's gradient (p - onehot) * scale for p = exp((z - M) k2) / S, by the nt threads of a group
// from thread t on; scale 0: zeros, without a look at the row.
template <typename T>
__device__ __forceinline__ void write_gradient(const RowSplit<T> &rs, T *drow, long long V, long long yv, float M,
                                               float S, float k2, float scale, long long t, long long nt) {
    using CV = Vec<T>;
    constexpr int EL = CV::ELEMS;
    const uint4 *src = reinterpret_cast<const uint4 *>(rs.row + rs.head);
    uint4 *dst = reinterpret_cast<uint4 *>(drow + rs.head);
    const long long extra = rs.head + (V - rs.tail0);
    if (scale == 0.f) {
        for (long long v = t; v < rs.nvec; v += nt) dst[v] = make_uint4(0u, 0u, 0u, 0u);
        if (t < extra) drow[rs.scalar(static_cast<int>(t), V)] = CV::from(0.f);
        return;
    }
    const ExpFrom e(M, k2);
    const float f = scale / S * e.c;
    const float2 f2 = make_float2(f, f);
    const long long yi = yv - rs.head;
    const long long vy = yv >= rs.head && yv < rs.tail0 ? yi / EL : -1;
    // the label's place is written again by the thread that wrote it; its logit is read before
    const bool mine = vy >= 0 ? vy >= t && vy < rs.nvec && (vy - t) % nt == 0
                              : t < extra && rs.scalar(static_cast<int>(t), V) == yv;
    const float zy = mine ? static_cast<float>(rs.row[yv]) : 0.f;
    auto one = [&](const uint4 &u, auto far) {
        uint4 out;
#pragma unroll
        for (int q = 0; q < CV::PAIRS; ++q) {
            const float2 z = CV::pair(u, q);
            CV::set_pair(out, q, __fmul2_rn(decltype(far)::value ? e.far_pair(z) : e.pair(z), f2));
        }
        return out;
    };
    long long v = t;
    if (e.far) {
#pragma unroll 1
        for (; v < rs.nvec; v += nt) dst[v] = one(src[v], std::true_type());
    }
    for (; v + 3 * nt < rs.nvec; v += 4 * nt) {
        uint4 u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = src[v + j * nt];
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[v + j * nt] = one(u[j], std::false_type());
    }
    for (; v < rs.nvec; v += nt) dst[v] = one(src[v], std::false_type());
    if (t < extra) {
        const long long i = rs.scalar(static_cast<int>(t), V);
        drow[i] = CV::from(e(static_cast<float>(rs.row[i])) * f);
    }
    if (mine) drow[yv] = CV::from(e(zy) * f - scale);
}

template <typename T>
__global__ void __launch_bounds__(STREAM_THREADS, 1) lce_answer_stream_kernel(const __grid_constant__ AnswerParams p) {
    using CV = Vec<T>;
    __shared__ float s_m[STREAM_THREADS / 32], s_s[STREAM_THREADS / 32];
    __shared__ float s_M, s_S, s_zy;
    __shared__ float2 s_red_d[STREAM_THREADS / 32];
    __shared__ int s_last;
    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    wait_for_previous_grid();
    const int nvalid = p.hdr[HDR_NVALID];
    const float k2 = LOG2E_F * p.pol.inv_t;
    for (long long r = blockIdx.x; r < p.N; r += gridDim.x) {
        const RowSplit<T> rs(static_cast<const T *>(p.Z) + r * p.ld, p.V);
        T *drow = p.dZ ? static_cast<T *>(p.dZ) + r * p.ld : nullptr;
        const long long yv = p.y[r];
        const bool y_ok = label_counts(yv, p.V, p.ignore_index);
        float scale = 0.f, M = 0.f, S = 1.f;
        if (y_ok) {
            if (t == 0) s_zy = static_cast<float>(rs.row[yv]);
            const uint4 *src = reinterpret_cast<const uint4 *>(rs.row + rs.head);
            float m = -INFINITY, s = 0.f;
            for (long long v = t; v < rs.nvec; v += STREAM_THREADS) {
                const uint4 u = src[v];
                const uint4 u1[1] = {u};
                const float mv = CV::max_of(u1, -INFINITY);
                const float nm = mv == -INFINITY ? 0.f : -mv;
                float sum = 0.f;
#pragma unroll
                for (int q = 0; q < CV::PAIRS; ++q) {
                    const float2 z = CV::pair(u, q);
                    sum += exp2_fast((z.x + nm) * k2) + exp2_fast((z.y + nm) * k2);
                }
                merge(m, s, mv, sum, k2);
            }
            const long long i = rs.scalar(t, p.V);
            if (i >= 0) {
                const float z = static_cast<float>(rs.row[i]);
                merge(m, s, z == z ? z : -INFINITY, z == z ? (z == -INFINITY ? 0.f : 1.f) : z, k2);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
                merge(m, s, m2, s2, k2);
            }
            if (l == 0) {
                s_m[w] = m;
                s_s[w] = s;
            }
            __syncthreads();
            if (w == 0) {
                m = s_m[l];
                s = s_s[l];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
                    merge(m, s, m2, s2, k2);
                }
                if (l == 0) {
                    s_M = m;
                    s_S = s;
                }
            }
            __syncthreads();
            M = s_M;
            S = s_S;
            const float logp = (s_zy - M) * p.pol.inv_t - logf(S);
            PolicyRow pr{-logp, 0.f};
            if (p.pol.adv) pr = lce_policy_row(p.pol, r, logp);
            scale = -pr.slope * p.pol.inv_t * lce_row_scale(p.dloss, p.dloss_per_row, p.mean, nvalid, r, true);
            if (t == 0) {
                p.loss_rows[r] = pr.loss;
                if (p.pol.logp) p.pol.logp[r] = logp;
            }
        } else if (t == 0) {
            p.loss_rows[r] = 0.f;
            if (p.pol.logp) p.pol.logp[r] = 0.f;
        }
        if (t == 0 && p.max_sum) p.max_sum[r] = make_float2(M, S);
        if (drow) write_gradient<T>(rs, drow, p.V, yv, M, S, k2, scale, t, STREAM_THREADS);
        __syncthreads();   // s_zy, s_M and the rest are used again
    }
    if (p.loss && last_to_finish(p.hdr + HDR_DONE, static_cast<int>(gridDim.x), &s_last)) write_loss(p, s_red_d);
}

// ------------------------------------------------------------------ the gradient of a preference
// Parts of rows, the last row first (its logits were read last and may still be in L2).

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_VECTORS = GRAD_THREADS * 8;   // of a part

template <typename T>
__global__ void __launch_bounds__(GRAD_THREADS) lce_answer_grad_kernel(const __grid_constant__ AnswerParams p,
                                                                       const int parts) {
    const long long r = p.N - 1 - static_cast<long long>(blockIdx.x) / parts;
    const long long part = static_cast<long long>(blockIdx.x) % parts;
    const RowSplit<T> rs(static_cast<const T *>(p.Z) + r * p.ld, p.V);
    T *drow = static_cast<T *>(p.dZ) + r * p.ld;
    const float2 ms = p.max_sum[r];
    RowSplit<T> mine = rs;   // the vectors of this part; the first part has the values beside them too
    const long long v0 = part * GRAD_VECTORS;
    mine.nvec = rs.nvec < v0 + GRAD_VECTORS ? rs.nvec : v0 + GRAD_VECTORS;
    // (written from vector v0 on: thread t starts at v0 + t)
    const long long first = v0 + threadIdx.x;
    write_gradient<T>(mine, drow, p.V, p.y[r], ms.x, ms.y, LOG2E_F, p.coef[r], first, GRAD_THREADS);
}

// ------------------------------------------------------------------ pairs

constexpr int PAIR_THREADS = 256;

__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A sequence's sum of log probabilities, what right label logits would add to it and the weight of that, and its
// counting rows.
struct Sequence {
    double sum, fix, weight;
    int rows;
};

// Of the rows begin .. end - 1, in every thread.
__device__ __forceinline__ Sequence sequence(const PairParams &p, long long begin, long long end, float2 *s_red,
                                             float2 *s_fix, int *s_cnt) {
    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    Sum2 s;
    float2 f = make_float2(0.f, 0.f);
    int n = 0;
    for (long long i = begin + t; i < end; i += PAIR_THREADS)
        if (label_counts(p.y[i], p.V, p.ignore_index)) {
            const long long at = p.place ? p.place[i] : i;
            s.add(-p.loss_rows[at]);
            if (p.fix) {
                const float2 x = p.fix[at];
                f.x += x.x;
                f.y += x.y;
            }
            ++n;
        }
    s.warp();
    f.x = lanes_sum(f.x);
    f.y = lanes_sum(f.y);
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (l == 0) {
        s_red[w] = make_float2(s.hi, s.lo);
        s_fix[w] = f;
        s_cnt[w] = n;
    }
    __syncthreads();
    const bool mine = l < PAIR_THREADS / 32;
    const float2 x = mine ? s_red[l] : make_float2(0.f, 0.f);
    f = mine ? s_fix[l] : make_float2(0.f, 0.f);
    s.hi = x.x;
    s.lo = x.y;
    s.warp();
    return Sequence{s.value(), lanes_sum(f.x), lanes_sum(f.y), __reduce_add_sync(0xffffffffu, mine ? s_cnt[l] : 0)};
}

// Offsets are taken as their running maximum, cut to [0, N]: whatever they hold, the sequences are disjoint and
// every row gets its coefficient. A pair's CTA looks through all offsets up to its own, which for many pairs is
// the square of their number: for more than PAIRS_BY_THEMSELVES one CTA forms the maxima before. (A call over 4000 x 64
// fp32 logits, replayed: 512 pairs 70 us without and 513 pairs 66 us with it, 2 pairs 60 without; 4096 pairs 297 us without and
// 107 with it, 100000 pairs 48.5 ms and 1.2 ms.)
constexpr int OFFS_THREADS = 1024, OFFS_EACH = 8;

__global__ void __launch_bounds__(OFFS_THREADS) lce_offsets_kernel(const long long *__restrict__ offsets, long long n,
                                                                   long long N, int *__restrict__ clean, int *hdr) {
    __shared__ int s_max[OFFS_THREADS / 32];
    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    bool bad = false;
    int before = 0;   // the maximum of the passes before (N fits 32 bits)
    for (long long base = 0; base < n; base += OFFS_THREADS * OFFS_EACH) {
        const long long i0 = base + static_cast<long long>(t) * OFFS_EACH;
        int v[OFFS_EACH], m = 0;
        long long last = i0 > 0 && i0 <= n ? offsets[i0 - 1] : 0;
#pragma unroll
        for (int j = 0; j < OFFS_EACH; ++j) {
            const long long o = i0 + j < n ? offsets[i0 + j] : last;
            bad |= i0 + j < n && (o < 0 || o > N || (i0 + j > 0 && o < last));
            last = o;
            m = max(m, i0 + j < n ? static_cast<int>(o < 0 ? 0 : o > N ? N : o) : 0);
            v[j] = m;
        }
        int up = m;   // of this thread and the lanes before it
#pragma unroll
        for (int s = 1; s < 32; s *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, up, s);
            if (l >= s) up = max(up, x);
        }
        if (l == 31) s_max[w] = up;
        __syncthreads();
        const int theirs = s_max[l];
        const int others = __reduce_max_sync(0xffffffffu, l < w ? theirs : 0);
        const int all = __reduce_max_sync(0xffffffffu, theirs);
        int lower = __shfl_up_sync(0xffffffffu, up, 1);
        lower = max(before, max(others, l > 0 ? lower : 0));
#pragma unroll
        for (int j = 0; j < OFFS_EACH; ++j)
            if (i0 + j < n) clean[i0 + j] = max(lower, v[j]);
        before = max(before, all);
        __syncthreads();
    }
    if (__syncthreads_or(bad) && t == 0) atomicOr(hdr + HDR_FLAG, FLAG_OFFSETS);
}

// One CTA per pair.
__global__ void __launch_bounds__(PAIR_THREADS) lce_pairs_kernel(const __grid_constant__ PairParams p) {
    __shared__ float2 s_red[PAIR_THREADS / 32], s_fix[PAIR_THREADS / 32];
    __shared__ int s_cnt[PAIR_THREADS / 32];
    __shared__ unsigned long long s_off[4];
    __shared__ int s_last;
    const int t = threadIdx.x;
    const long long k = blockIdx.x;
    const long long want[4] = {k, k + 1, p.pairs + k, p.pairs + k + 1};
    if (t < 4) s_off[t] = 0;
    __syncthreads();
    bool bad = false;
    if (p.clean && t < 4) s_off[t] = p.clean[want[t]];
    for (long long i = t; !p.clean && i <= p.pairs + k + 1; i += PAIR_THREADS) {
        const long long o = p.offsets[i];
        bad |= o < 0 || o > p.N || (i > 0 && o < p.offsets[i - 1]);
        const unsigned long long c = o < 0 ? 0 : o > p.N ? p.N : o;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (i <= want[q]) atomicMax(&s_off[q], c);
    }
    if (__syncthreads_or(bad) && t == 0) atomicOr(p.hdr + HDR_FLAG, FLAG_OFFSETS);
    const long long off[4] = {static_cast<long long>(s_off[0]), static_cast<long long>(s_off[1]),
                              static_cast<long long>(s_off[2]), static_cast<long long>(s_off[3])};
    double sum[2];
    int n[2];
    const Sequence chosen = sequence(p, off[0], off[1], s_red, s_fix, s_cnt);
    const Sequence rejected = sequence(p, off[2], off[3], s_red, s_fix, s_cnt);
    sum[0] = chosen.sum;
    sum[1] = rejected.sum;
    n[0] = chosen.rows;
    n[1] = rejected.rows;
    // Over the head, the tensor cores cut their sums over D after each step: a logit z is off by about -3.5e-6 z at D =
    // 4096, lse by the same on average over what the model would draw, and each row's log probability by 1.4e-5 rms
    // of z_y's share in it, which sums over hundreds of rows and the margin keep. A right z_y alone
    // would leave lse's part (-3.5e-5 a row, all of one sign). So z_y is put right but for the mean over the
    // pair's rows, which is the part that lse has too; the pair's log probabilities add up to what they did.
    const double weight = chosen.weight + rejected.weight, both = chosen.fix + rejected.fix;
    if (weight > 0.0) {
        const double fix[2] = {chosen.fix - both / weight * chosen.weight, rejected.fix - both / weight * rejected.weight};
        for (int q = 0; q < 2; ++q)
            if (fabs(fix[q]) < INFINITY) sum[q] += fix[q];
    }
    float share[2];
    for (int q = 0; q < 2; ++q) {
        share[q] = p.average && n[q] > 0 ? 1.f / static_cast<float>(n[q]) : 1.f;
        if (p.average && n[q] > 0) sum[q] /= n[q];
    }
    // the loss of the margin and its slope:
    //   m = beta ((L_c - R_c) - (L_r - R_r)), loss = -((1 - e) log sig(m) + e log sig(-m))
    //   d loss / d L_c = beta (e sig(m) - (1 - e) sig(-m)) = - d loss / d L_r
    // (the differences in fp64: sums of hundreds of log probabilities nearly cancel)
    const double rc = p.ref ? p.ref[k] : 0.f, rr = p.ref ? p.ref[p.pairs + k] : 0.f;
    const float m = static_cast<float>(p.beta * ((sum[0] - rc) - (sum[1] - rr))), e = p.smoothing;
    const float tail = log1pf(expf(-fabsf(m)));
    const float log_right = fminf(m, 0.f) - tail, log_wrong = fminf(-m, 0.f) - tail;
    float loss = -(1.f - e) * log_right;
    if (e > 0.f) loss -= e * log_wrong;
    if (m != m) loss = m;   // (fminf drops a NaN)
    if (t == 0) {
        p.seq_logp[k] = static_cast<float>(sum[0]);
        p.seq_logp[p.pairs + k] = static_cast<float>(sum[1]);
        p.pair_loss[k] = static_cast<float>(loss);
    }
    if (p.coef) {
        float d = p.dloss ? p.dloss[p.dloss_per_pair ? k : 0] : 1.f;
        if (p.mean) d /= static_cast<float>(p.pairs);
        const float big = 1.f / (1.f + expf(-fabsf(m))), small = expf(-fabsf(m)) * big;   // sigmoids
        float slope = p.beta * (e * (m >= 0.f ? big : small) - (1.f - e) * (m >= 0.f ? small : big)) * d;
        if (m != m) slope = m;
        // p - onehot gets minus the slope of its row
        const float c[2] = {-slope * share[0], slope * share[1]};
        auto put = [&](long long i, float v) {
            const long long at = p.place ? p.place[i] : i;
            if (at >= 0) p.coef[at] = v;
        };
        for (int q = 0; q < 2; ++q)
            for (long long i = off[2 * q] + t; i < off[2 * q + 1]; i += PAIR_THREADS)
                put(i, label_counts(p.y[i], p.V, p.ignore_index) ? c[q] : 0.f);
        // rows before the first sequence and behind the last
        if (k == 0)
            for (long long i = t; i < p.N && i < off[0]; i += PAIR_THREADS) put(i, 0.f);
        if (k == p.pairs - 1)
            for (long long i = off[3] + t; i < p.N; i += PAIR_THREADS) put(i, 0.f);
    }
    if (p.loss && last_to_finish(p.hdr + HDR_DONE, static_cast<int>(gridDim.x), &s_last)) {
        const double s = block_sum(p.pair_loss, p.pairs, s_red);
        if (t == 0) *p.loss = static_cast<float>(p.mean ? s / static_cast<double>(p.pairs) : s);
    }
}

// ------------------------------------------------------------------ scaled gradients
// Eight values per thread and step, where both places start on 16 bytes; else one.

constexpr int SCALE_THREADS = 256;

template <typename S, typename D>
__global__ void __launch_bounds__(SCALE_THREADS) lce_scale_kernel(const S *src, const float *__restrict__ scale,
                                                                  long long n, D *dst, int vec) {
    const float g = *scale;
    if (g == 1.f && static_cast<const void *>(src) == static_cast<const void *>(dst)) return;   // (they are that already)
    const long long t = blockIdx.x * static_cast<long long>(SCALE_THREADS) + threadIdx.x;
    const long long nt = static_cast<long long>(gridDim.x) * SCALE_THREADS;
    const long long nv = vec ? n / 8 : 0;
    constexpr int SV = 8 / Vec<S>::ELEMS, DV = 8 / Vec<D>::ELEMS;   // 16-byte vectors of eight values
#pragma unroll 4
    for (long long i = t; i < nv; i += nt) {
        float2 x[4];
#pragma unroll
        for (int j = 0; j < SV; ++j) {
            const uint4 u = reinterpret_cast<const uint4 *>(src)[i * SV + j];
#pragma unroll
            for (int q = 0; q < Vec<S>::PAIRS; ++q) x[j * Vec<S>::PAIRS + q] = Vec<S>::pair(u, q);
        }
#pragma unroll
        for (int j = 0; j < DV; ++j) {
            uint4 u;
#pragma unroll
            for (int q = 0; q < Vec<D>::PAIRS; ++q) {
                const float2 v = x[j * Vec<D>::PAIRS + q];
                Vec<D>::set_pair(u, q, make_float2(v.x * g, v.y * g));
            }
            reinterpret_cast<uint4 *>(dst)[i * DV + j] = u;
        }
    }
    for (long long i = nv * 8 + t; i < n; i += nt) dst[i] = Vec<D>::from(static_cast<float>(src[i]) * g);
}

// ------------------------------------------------------------------ launches

using RowsKernel = void (*)(const AnswerParams, const int, const int);

RowsKernel rows_kernel(int dtype) {
    return dtype == CE_FP32 ? lce_answer_rows_kernel<float>
           : dtype == CE_FP16 ? lce_answer_rows_kernel<__half> : lce_answer_rows_kernel<__nv_bfloat16>;
}

int g_ans_max_dyn[64];   // per device: dynamic shared memory the cluster kernel may take

struct Shape {
    int cl = 0, sv = 0, nbuf = 0;
    size_t smem = 0;
};

// The smallest cluster of whose rows three buffers fit into a CTA's shared memory, else two; with
// so few rows that SMs would idle, a larger one.
bool rows_shape(const AnswerParams &p, int sms, int max_dyn, Shape *o) {
    const long long nvec = p.V / (p.dtype == CE_FP32 ? 4 : 8);
    auto bytes = [&](int cl) { return ((nvec + cl - 1) / cl > 0 ? (nvec + cl - 1) / cl : 1) * 16; };
    int cl = 1;
    while (cl < ANS_MAX_CLUSTER && 3 * bytes(cl) > max_dyn) cl *= 2;
    if (2 * bytes(cl) > max_dyn) return false;
    while (cl < ANS_MAX_CLUSTER && p.N * cl * 2 <= sms && nvec / cl > ANS_THREADS) cl *= 2;
    o->cl = cl;
    o->sv = static_cast<int>(bytes(cl) / 16);
    o->nbuf = max_dyn / bytes(cl) < ANS_MAX_BUF ? 2 : ANS_MAX_BUF;
    o->smem = o->nbuf * static_cast<size_t>(bytes(cl));
    return true;
}

std::mutex g_ans_mu;
std::map<long long, int> g_ans_occ;   // (device, kernel, cluster, smem) -> co-resident clusters

cudaLaunchAttribute after_previous() {
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

cudaError_t launch_rows_cluster(const AnswerParams &p, const Shape &sh, int dev, bool *launched, cudaStream_t s) {
    *launched = false;
    const RowsKernel fn = rows_kernel(p.dtype);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = sh.cl;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1] = after_previous();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.cl);
    cfg.blockDim = dim3(ANS_THREADS + 64);
    cfg.dynamicSmemBytes = sh.smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const long long key = ((static_cast<long long>(dev) * 4 + p.dtype) * 16 + sh.cl) * (1ll << 24) +
                          static_cast<long long>(sh.smem);
    int n = -1;
    {
        std::lock_guard<std::mutex> lock(g_ans_mu);
        auto f = g_ans_occ.find(key);
        if (f != g_ans_occ.end()) n = f->second;
    }
    if (n < 0) {
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        std::lock_guard<std::mutex> lock(g_ans_mu);
        g_ans_occ[key] = n;
    }
    if (n <= 0) return cudaSuccess;   // the caller streams
    cfg.gridDim = dim3(static_cast<unsigned>((n < p.N ? n : p.N) * sh.cl));
    cfg.numAttrs = 2;
    *launched = true;
    return cudaLaunchKernelEx(&cfg, fn, p, sh.sv, sh.nbuf);
}

template <typename T> cudaError_t launch_rows_stream(const AnswerParams &p, int sms, cudaStream_t s) {
    cudaLaunchAttribute at[1] = {after_previous()};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.N < sms ? p.N : sms));
    cfg.blockDim = dim3(STREAM_THREADS);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lce_answer_stream_kernel<T>, p);
}

template <typename T> cudaError_t launch_grad_of(const AnswerParams &p, cudaStream_t s) {
    const long long parts = (p.V / Vec<T>::ELEMS + GRAD_VECTORS - 1) / GRAD_VECTORS;
    const int np = parts < 1 ? 1 : static_cast<int>(parts);
    if (p.N * np > 0x7fffffffll) return cudaErrorInvalidValue;
    lce_answer_grad_kernel<T><<<static_cast<unsigned>(p.N * np), GRAD_THREADS, 0, s>>>(p, np);
    return cudaGetLastError();
}

template <typename S, typename D>
cudaError_t launch_scale_of(const void *src, const float *scale, long long n, void *dst, int sms, cudaStream_t s) {
    const int vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u) == 0;
    long long blocks = (n / (vec ? 8 : 1) + SCALE_THREADS - 1) / SCALE_THREADS;
    if (blocks > 16ll * sms) blocks = 16ll * sms;
    if (blocks < 1) blocks = 1;
    lce_scale_kernel<S, D><<<static_cast<unsigned>(blocks), SCALE_THREADS, 0, s>>>(
        static_cast<const S *>(src), scale, n, static_cast<D *>(dst), vec);
    return cudaGetLastError();
}
template <typename S>
cudaError_t launch_scale_from(const void *src, const float *scale, long long n, void *dst, int dst_dtype, int sms,
                              cudaStream_t s) {
    return dst_dtype == CE_FP32 ? launch_scale_of<S, float>(src, scale, n, dst, sms, s)
           : dst_dtype == CE_FP16 ? launch_scale_of<S, __half>(src, scale, n, dst, sms, s)
                                  : launch_scale_of<S, __nv_bfloat16>(src, scale, n, dst, sms, s);
}

}  // namespace

cudaError_t answers_set_attributes() {
    int dev = 0, optin = 0, used = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return e;
    for (int pass = 0; pass < 2; ++pass)
        for (int dt = 0; dt < 3; ++dt) {
            if (pass == 0) {
                cudaFuncAttributes fa{};
                e = cudaFuncGetAttributes(&fa, rows_kernel(dt));
                if (static_cast<int>(fa.sharedSizeBytes) > used) used = static_cast<int>(fa.sharedSizeBytes);
            } else {
                e = cudaFuncSetAttribute(rows_kernel(dt), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         optin - used - 1024);
            }
            if (e != cudaSuccess) return e;
        }
    g_ans_max_dyn[dev] = optin - used - 1024;
    return cudaSuccess;
}

cudaError_t launch_answer_scan(const long long *y, long long N, long long V, long long ign, int *hdr,
                               cudaStream_t s) {
    if (N > SCAN_ONE_CTA) {
        const cudaError_t e = cudaMemsetAsync(hdr, 0, 4 * HDR_COUNTERS, s);
        return e != cudaSuccess ? e : launch_label_scan(y, N, V, ign, hdr, s);
    }
    lce_answer_scan_kernel<<<1, 1024, 0, s>>>(y, N, V, ign, hdr);
    return cudaGetLastError();
}

cudaError_t launch_answer_rows(const AnswerParams &p, int sms, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    Shape sh;
    if (dev >= 0 && dev < 64 && rows_shape(p, sms, g_ans_max_dyn[dev], &sh)) {
        bool launched = false;
        e = launch_rows_cluster(p, sh, dev, &launched, s);
        if (e != cudaSuccess || launched) return e;
    }
    return p.dtype == CE_FP32 ? launch_rows_stream<float>(p, sms, s)
           : p.dtype == CE_FP16 ? launch_rows_stream<__half>(p, sms, s) : launch_rows_stream<__nv_bfloat16>(p, sms, s);
}

cudaError_t launch_answer_grad(const AnswerParams &p, int, cudaStream_t s) {
    return p.dtype == CE_FP32 ? launch_grad_of<float>(p, s)
           : p.dtype == CE_FP16 ? launch_grad_of<__half>(p, s) : launch_grad_of<__nv_bfloat16>(p, s);
}

cudaError_t launch_offsets(const PairParams &p, cudaStream_t s) {
    lce_offsets_kernel<<<1, OFFS_THREADS, 0, s>>>(p.offsets, 2 * p.pairs + 1, p.N, p.clean, p.hdr);
    return cudaGetLastError();
}

cudaError_t launch_pairs(const PairParams &p, cudaStream_t s) {
    lce_pairs_kernel<<<static_cast<unsigned>(p.pairs), PAIR_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_scale(const void *src, int src_dtype, const float *scale, long long n, void *dst, int dst_dtype,
                         int sms, cudaStream_t s) {
    return src_dtype == CE_FP32 ? launch_scale_from<float>(src, scale, n, dst, dst_dtype, sms, s)
           : src_dtype == CE_FP16 ? launch_scale_from<__half>(src, scale, n, dst, dst_dtype, sms, s)
                                  : launch_scale_from<__nv_bfloat16>(src, scale, n, dst, dst_dtype, sms, s);
}

}  // namespace lce
