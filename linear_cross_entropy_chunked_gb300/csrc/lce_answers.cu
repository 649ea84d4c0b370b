// Losses on answers: what the log probabilities of drawn tokens are worth, and the gradient.
//
//   * rows of given logits: log p of the row's label, the clipped policy loss with its KL term
//     and the gradient (p - onehot) * scale in one pass over the logits (cluster kernel), or
//     in two for rows beyond eight CTAs' registers (streaming kernel);
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
constexpr int ANS_MAX_VPT = 16;                  // 16-byte vectors per thread
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
    __device__ static float max2(const uint4 &u, float m) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
        const __nv_bfloat162 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
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
    __device__ static float max2(const uint4 &u, float m) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&u);
        const __half2 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
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
    __device__ static float max2(const uint4 &u, float m) {
        return fmaxf(fmaxf(m, fmaxf(__uint_as_float(u.x), __uint_as_float(u.y))),
                     fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
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
// A cluster of 1 to 8 CTAs takes one row at a time; rank k owns the vectors [k sv, (k + 1) sv)
// of it, rank 0 also the values beside them (one per thread). Per row, in each CTA:
//   * bulk copies have brought the vectors into a buffer; the threads move theirs into
//     registers, whereupon the buffer is filled again with the row nbuf steps ahead;
//   * max, then the sum of exp((z - max) / T);
//   * (max, sum, label's logit if it lies here) goes to every CTA of the cluster by st.async;
//   * the label's log probability, the row's loss and its slope, in every thread; the gradient
//     exp((z - max) / T) * (scale / sum) - onehot * scale from the registers. The exponentials are
//     formed again, not kept: they are the very numbers that were summed, and 16-bit logits would
//     have to round them.

template <typename T, int VPT>
__global__ void __launch_bounds__(ANS_THREADS, 1)
    lce_answer_rows_kernel(const __grid_constant__ AnswerParams p, const int sv, const int nbuf) {
    using CV = Vec<T>;
    constexpr int EL = CV::ELEMS;
    extern __shared__ __align__(128) uint8_t ans_smem[];
    __shared__ __align__(8) uint64_t lbar[ANS_MAX_BUF];    // a row's copies landed
    __shared__ __align__(8) uint64_t xbar[2];              // every CTA's (max, sum, logit) landed
    __shared__ __align__(16) float4 xslot[2][ANS_MAX_CLUSTER];
    __shared__ float s_red_m[ANS_WARPS], s_red_s[ANS_WARPS];
    __shared__ float2 s_red_d[ANS_WARPS];
    __shared__ int s_abort, s_last;

    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    const uint32_t rank = cluster_ctarank(), cl = cluster_ctas();
    const long long cid = cluster_id(), ncl = cluster_count();
    const Abort ab{&s_abort, p.hdr, ANS_WAIT_NS};
    const T *Z = static_cast<const T *>(p.Z);

    if (t == 0) {
        s_abort = 0;
        for (int b = 0; b < nbuf; ++b) mbar_init(&lbar[b], 1);
        mbar_init(&xbar[0], 1);
        mbar_init(&xbar[1], 1);
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
    // thread 0: starts the copies of the cluster's it-th row, whose label is yi, into buffer b
    long long issued = 0;
    auto issue = [&](long long it, int b, long long yi) {
        const long long r = cid + it * ncl;
        if (r >= p.N) return;
        issued = it + 1;
        const RowSplit<T> rs(Z + r * p.ld, p.V);
        const uint32_t bytes = label_counts(yi, p.V, p.ignore_index) ? vectors(rs) * 16u : 0u;
        if (bytes == 0) {
            mbar_arrive(&lbar[b]);
            return;
        }
        mbar_arrive_expect_tx(&lbar[b], bytes);
        const uint8_t *src = reinterpret_cast<const uint8_t *>(rs.row + rs.head + v0 * EL);
        const uint32_t dst = smem_u32(ans_smem + static_cast<size_t>(b) * sv * 16);
        for (uint32_t off = 0; off < bytes; off += ANS_COPY_BYTES)
            bulk_copy(dst + off, src + off, bytes - off < ANS_COPY_BYTES ? bytes - off : ANS_COPY_BYTES,
                      smem_u32(&lbar[b]));
    };
    auto label = [&](long long it) -> long long {
        const long long r = cid + it * ncl;
        return r < p.N ? p.y[r] : p.ignore_index;
    };
    long long y_ahead = 0;   // thread 0: the label of the row that is issued next
    if (t == 0) {
        for (int j = 0; j < nbuf; ++j) issue(j, j, label(j));
        y_ahead = label(nbuf);
    }

    wait_for_previous_grid();   // the header
    const int nvalid = p.hdr[HDR_NVALID];
    const float k2 = LOG2E_F * p.pol.inv_t;
    const float2 kk = make_float2(k2, k2);
    int buf = 0, xs = 0;
    uint32_t lpar = 0, xpar = 0;
    bool bad = false, aborted = false;
    long long it = 0, y_next = label(0);
    for (; cid + it * ncl < p.N; ++it) {
        const long long r = cid + it * ncl;
        const long long yv = y_next;
        y_next = label(it + 1);
        const RowSplit<T> rs(Z + r * p.ld, p.V);
        const int nvec = vectors(rs);
        const bool y_ok = label_counts(yv, p.V, p.ignore_index);
        T *drow = p.dZ ? static_cast<T *>(p.dZ) + r * p.ld : nullptr;
        uint4 *dvec = reinterpret_cast<uint4 *>(drow + rs.head) + v0;   // (not used where dZ is null)
        const long long si = rank == 0 ? rs.scalar(t, p.V) : -1;
        bad |= !mbar_wait(&lbar[buf], lpar, ab);
        if (!y_ok) {
            // every thread has seen this phase of the buffer's barrier before it can go on by two more
            if (__syncthreads_or(bad)) {
                aborted = true;
                break;
            }
            if (t == 0) {
                issue(it + nbuf, buf, y_ahead);
                y_ahead = label(it + nbuf + 1);
                if (rank == 0) {
                    p.loss_rows[r] = 0.f;
                    if (p.pol.logp) p.pol.logp[r] = 0.f;
                    if (p.max_sum) p.max_sum[r] = make_float2(0.f, 1.f);
                }
            }
            if (drow) {
                for (int v = t; v < nvec; v += ANS_THREADS) dvec[v] = make_uint4(0u, 0u, 0u, 0u);
                if (si >= 0) drow[si] = CV::from(0.f);
            }
        } else {
            const uint4 *sg = reinterpret_cast<const uint4 *>(ans_smem + static_cast<size_t>(buf) * sv * 16);
            // where the label's logit lies: in a vector of this CTA, or beside the vectors (rank 0)
            const long long yi = yv - rs.head - v0 * EL;
            const bool in_vec = yv >= rs.head && yv < rs.tail0;
            const int yl = in_vec && yi >= 0 && yi < static_cast<long long>(nvec) * EL ? static_cast<int>(yi) : -1;
            uint4 d[VPT];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = t + k * ANS_THREADS;
                d[k] = v < nvec ? sg[v] : make_uint4(CV::NEG_INF, CV::NEG_INF, CV::NEG_INF, CV::NEG_INF);
            }
            const float xsc = si >= 0 ? static_cast<float>(rs.row[si]) : -INFINITY;
            float zy = 0.f;
            if (t == 0) {
                if (yl >= 0) zy = static_cast<float>(reinterpret_cast<const T *>(sg)[yl]);
                else if (rank == 0 && !in_vec) zy = static_cast<float>(rs.row[yv]);
                mbar_arrive_expect_tx(&xbar[xs], cl * 16u);
            }
            float m = xsc;
#pragma unroll
            for (int k = 0; k < VPT; ++k) m = CV::max2(d[k], m);
            m = wmax(m);
            if (l == 0) s_red_m[w] = m;
            // every thread holds its vectors: the buffer may be filled again; also the abort vote
            if (__syncthreads_or(bad)) {
                aborted = true;
                break;
            }
            if (t == 0) {
                fence_proxy_async_smem();
                issue(it + nbuf, buf, y_ahead);
                y_ahead = label(it + nbuf + 1);
            }
            m = wmax(l < ANS_WARPS ? s_red_m[l] : -INFINITY);
            // (the distance from the maximum first: its product with k2 may be beyond fp32, as for a row
            // of the type's lowest value; with nothing here every exponential is 0)
            const float nm = m == -INFINITY ? 0.f : -m;
            const float2 nm2 = make_float2(nm, nm);
            float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int q = 0; q < CV::PAIRS; ++q) {
                    const float2 a = __fmul2_rn(__fadd2_rn(CV::pair(d[k], q), nm2), kk);
                    const float2 e = make_float2(exp2_fast(a.x), exp2_fast(a.y));
                    if (q & 1) acc1 = __fadd2_rn(acc1, e);
                    else acc0 = __fadd2_rn(acc0, e);
                }
            const float2 acc = __fadd2_rn(acc0, acc1);
            float s = wsum(acc.x + acc.y + exp2_fast((xsc + nm) * k2));
            if (l == 0) s_red_s[w] = s;
            __syncthreads();
            s = wsum(l < ANS_WARPS ? s_red_s[l] : 0.f);
            zy = __shfl_sync(0xffffffffu, zy, 0);   // (warp 0 sends: its lane 0 has it)
            if (w == 0 && l < static_cast<int>(cl))
                st_async_f32x4(map_to_rank(&xslot[xs][rank], l), m, s, zy, 0.f, map_to_rank(&xbar[xs], l));
            const bool xok = mbar_wait_cluster(&xbar[xs], xpar, ab);
            bad |= !xok;
            if (xok) {
                // lane k holds rank k's part; the maximum, the sum in rank order, the one logit
                const float4 x = l < static_cast<int>(cl) ? xslot[xs][l] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
                float M = x.x;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                float S = x.x == -INFINITY ? x.y : x.y * exp2f((x.x - M) * k2);   // (0, or a NaN)
                float zl = x.z;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) {
                    S += __shfl_xor_sync(0xffffffffu, S, o);
                    zl += __shfl_xor_sync(0xffffffffu, zl, o);
                }
                M = __shfl_sync(0xffffffffu, M, 0);
                S = __shfl_sync(0xffffffffu, S, 0);
                zl = __shfl_sync(0xffffffffu, zl, 0);
                const float logp = (zl - M) * p.pol.inv_t - logf(S);
                PolicyRow pr{-logp, 0.f};
                if (p.pol.adv) pr = lce_policy_row(p.pol, r, logp);
                if (t == 0 && rank == 0) {
                    p.loss_rows[r] = pr.loss;
                    if (p.pol.logp) p.pol.logp[r] = logp;
                    if (p.max_sum) p.max_sum[r] = make_float2(M, S);
                }
                if (drow) {
                    const float scale = -pr.slope * p.pol.inv_t *
                                        lce_row_scale(p.dloss, p.dloss_per_row, p.mean, nvalid, r, true);
                    if (scale == 0.f) {
                        for (int v = t; v < nvec; v += ANS_THREADS) dvec[v] = make_uint4(0u, 0u, 0u, 0u);
                        if (si >= 0) drow[si] = CV::from(0.f);
                    } else {
                        const float f = (m == -INFINITY ? 1.f : exp2f((m - M) * k2)) * (scale / S);
                        const float2 f2 = make_float2(f, f);
                        const int vy = yl >= 0 ? yl / EL : -1, jy = yl & (EL - 1);
#pragma unroll
                        for (int k = 0; k < VPT; ++k) {
                            const int v = t + k * ANS_THREADS;
                            if (v < nvec) {
                                uint4 out;
#pragma unroll
                                for (int q = 0; q < CV::PAIRS; ++q) {
                                    const float2 a = __fmul2_rn(__fadd2_rn(CV::pair(d[k], q), nm2), kk);
                                    float2 g = __fmul2_rn(make_float2(exp2_fast(a.x), exp2_fast(a.y)), f2);
                                    if (v == vy) {
                                        if (2 * q == jy) g.x -= scale;
                                        if (2 * q + 1 == jy) g.y -= scale;
                                    }
                                    CV::set_pair(out, q, g);
                                }
                                dvec[v] = out;
                            }
                        }
                        if (si >= 0) {
                            float g = exp2_fast((xsc + nm) * k2) * f;
                            if (si == yv) g -= scale;
                            drow[si] = CV::from(g);
                        }
                    }
                }
            }
            xs ^= 1;
            if (xs == 0) xpar ^= 1u;
        }
        if (++buf == nbuf) {
            buf = 0;
            lpar ^= 1u;
        }
    }
    aborted = __syncthreads_or(aborted || bad);
    if (aborted && t == 0)
        // copies of rows it .. issued - 1 may still be landing here
        for (long long j = it; j < issued; ++j)
            mbar_wait_drain(&lbar[j % nbuf], static_cast<uint32_t>((j / nbuf) & 1), ANS_WAIT_NS);
    __syncthreads();
    cluster_sync_all();   // no CTA leaves while a peer may still write into its slots
    if (rank == 0 && p.loss && last_to_finish(p.hdr + HDR_DONE, static_cast<int>(ncl), &s_last))
        write_loss(p, s_red_d);
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
    const float nm = -M, f = scale / S;
    const float2 kk = make_float2(k2, k2), nm2 = make_float2(nm, nm), f2 = make_float2(f, f);
    const long long yi = yv - rs.head;
    const long long vy = yv >= rs.head && yv < rs.tail0 ? yi / EL : -1;
    const int jy = static_cast<int>(yi & (EL - 1));
    auto one = [&](long long v, const uint4 &u) {
        uint4 out;
#pragma unroll
        for (int q = 0; q < CV::PAIRS; ++q) {
            const float2 a = __fmul2_rn(__fadd2_rn(CV::pair(u, q), nm2), kk);
            float2 g = __fmul2_rn(make_float2(exp2_fast(a.x), exp2_fast(a.y)), f2);
            if (v == vy) {
                if (2 * q == jy) g.x -= scale;
                if (2 * q + 1 == jy) g.y -= scale;
            }
            CV::set_pair(out, q, g);
        }
        dst[v] = out;
    };
    long long v = t;
    for (; v + 3 * nt < rs.nvec; v += 4 * nt) {
        uint4 u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = src[v + j * nt];
#pragma unroll
        for (int j = 0; j < 4; ++j) one(v + j * nt, u[j]);
    }
    for (; v < rs.nvec; v += nt) one(v, src[v]);
    if (t < extra) {
        const long long i = rs.scalar(static_cast<int>(t), V);
        float g = exp2_fast((static_cast<float>(rs.row[i]) + nm) * k2) * f;
        if (i == yv) g -= scale;
        drow[i] = CV::from(g);
    }
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
                const float mv = CV::max2(u, -INFINITY);
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

// Sum and count of the counting rows begin .. end - 1, in every thread.
__device__ __forceinline__ void sequence(const PairParams &p, long long begin, long long end, float2 *s_red,
                                         int *s_cnt, double *sum, int *count) {
    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    Sum2 s;
    int n = 0;
    for (long long i = begin + t; i < end; i += PAIR_THREADS)
        if (label_counts(p.y[i], p.V, p.ignore_index)) {
            s.add(-p.loss_rows[i]);
            ++n;
        }
    s.warp();
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (l == 0) {
        s_red[w] = make_float2(s.hi, s.lo);
        s_cnt[w] = n;
    }
    __syncthreads();
    const float2 x = l < PAIR_THREADS / 32 ? s_red[l] : make_float2(0.f, 0.f);
    s.hi = x.x;
    s.lo = x.y;
    s.warp();
    *sum = s.value();
    *count = __reduce_add_sync(0xffffffffu, l < PAIR_THREADS / 32 ? s_cnt[l] : 0);
}

// One CTA per pair. Offsets are taken as their running maximum, cut to [0, N]: whatever they
// hold, the sequences are disjoint and every row gets its coefficient.
__global__ void __launch_bounds__(PAIR_THREADS) lce_pairs_kernel(const __grid_constant__ PairParams p) {
    __shared__ float2 s_red[PAIR_THREADS / 32];
    __shared__ int s_cnt[PAIR_THREADS / 32];
    __shared__ unsigned long long s_off[4];
    __shared__ int s_last;
    const int t = threadIdx.x;
    const long long k = blockIdx.x;
    const long long want[4] = {k, k + 1, p.pairs + k, p.pairs + k + 1};
    if (t < 4) s_off[t] = 0;
    __syncthreads();
    bool bad = false;
    for (long long i = t; i <= p.pairs + k + 1; i += PAIR_THREADS) {
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
    sequence(p, off[0], off[1], s_red, s_cnt, &sum[0], &n[0]);
    sequence(p, off[2], off[3], s_red, s_cnt, &sum[1], &n[1]);
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
        for (int q = 0; q < 2; ++q)
            for (long long i = off[2 * q] + t; i < off[2 * q + 1]; i += PAIR_THREADS)
                p.coef[i] = label_counts(p.y[i], p.V, p.ignore_index) ? c[q] : 0.f;
        // rows before the first sequence and behind the last
        if (k == 0)
            for (long long i = t; i < p.N; i += PAIR_THREADS)
                if (i < off[0]) p.coef[i] = 0.f;
                else break;
        if (k == p.pairs - 1)
            for (long long i = off[3] + t; i < p.N; i += PAIR_THREADS) p.coef[i] = 0.f;
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

template <typename T> RowsKernel rows_kernel_of(int vpt) {
    switch (vpt) {
        case 1: return lce_answer_rows_kernel<T, 1>;
        case 2: return lce_answer_rows_kernel<T, 2>;
        case 4: return lce_answer_rows_kernel<T, 4>;
        case 8: return lce_answer_rows_kernel<T, 8>;
        default: return lce_answer_rows_kernel<T, 16>;
    }
}
RowsKernel rows_kernel(int dtype, int vpt) {
    return dtype == CE_FP32 ? rows_kernel_of<float>(vpt)
           : dtype == CE_FP16 ? rows_kernel_of<__half>(vpt) : rows_kernel_of<__nv_bfloat16>(vpt);
}

int g_ans_max_dyn[64];   // per device: dynamic shared memory the cluster kernel may take

struct Shape {
    int cl = 0, sv = 0, vpt = 0, nbuf = 0;
    size_t smem = 0;
};

// The smallest cluster whose CTAs hold a row in registers; with so few rows that SMs would
// idle, a larger one.
bool rows_shape(const AnswerParams &p, int sms, int max_dyn, Shape *o) {
    const long long el = p.dtype == CE_FP32 ? 4 : 8;
    const long long nvec = p.V / el;
    int cl = 1;
    while (cl <= ANS_MAX_CLUSTER && (nvec + cl - 1) / cl > ANS_THREADS * ANS_MAX_VPT) ++cl;
    if (cl > ANS_MAX_CLUSTER) return false;
    while (cl < ANS_MAX_CLUSTER && p.N * cl * 2 <= sms && nvec / cl > ANS_THREADS) cl *= 2;
    if (cl > ANS_MAX_CLUSTER) cl = ANS_MAX_CLUSTER;
    o->cl = cl;
    o->sv = static_cast<int>((nvec + cl - 1) / cl);
    if (o->sv < 1) o->sv = 1;
    o->vpt = 1;
    while (ANS_THREADS * o->vpt < o->sv) o->vpt *= 2;
    const size_t bytes = static_cast<size_t>(o->sv) * 16;
    const long long fit = max_dyn / static_cast<long long>(bytes);
    if (fit < 1) return false;
    o->nbuf = fit < ANS_MAX_BUF ? static_cast<int>(fit) : ANS_MAX_BUF;
    o->smem = o->nbuf * bytes;
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
    const RowsKernel fn = rows_kernel(p.dtype, sh.vpt);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = sh.cl;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1] = after_previous();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.cl);
    cfg.blockDim = dim3(ANS_THREADS);
    cfg.dynamicSmemBytes = sh.smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const long long key = (((static_cast<long long>(dev) * 4 + p.dtype) * 32 + sh.vpt) * 16 + sh.cl) * (1ll << 24) +
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
        for (int dt = 0; dt < 3; ++dt)
            for (int vpt = 1; vpt <= ANS_MAX_VPT; vpt *= 2) {
                if (pass == 0) {
                    cudaFuncAttributes fa{};
                    e = cudaFuncGetAttributes(&fa, rows_kernel(dt, vpt));
                    if (static_cast<int>(fa.sharedSizeBytes) > used) used = static_cast<int>(fa.sharedSizeBytes);
                } else {
                    e = cudaFuncSetAttribute(rows_kernel(dt, vpt), cudaFuncAttributeMaxDynamicSharedMemorySize,
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
