// The global norm of a list of gradients (bf16, fp16 or fp32, mixed), and clipping by it:
//   norm = (sum over all values of |g|^p)^(1/p), p = 1 or 2, or max |g|
//   g <- g * min(1, max_norm / (norm + eps))
//
// Two launches per list (more only beyond CLIP_MAX_TENSORS tensors), bound by HBM
// bandwidth: one read for the norm, and one read and one write for the scaling, which
// leaves at once where the factor is 1 and the values stay where they are. The list
// travels in the kernels' parameters, so nothing is copied to the device first and a
// captured graph keeps it.
//
// A launch cuts every tensor into chunks of CLIP_CHUNK bytes; CTA b takes chunks b, b + grid,
// ... With a run of consecutive chunks per CTA the norm and scaling of 2.1 GB of fp32 into
// another buffer took 1.18 ms; so it takes 1.00 ms, the norm at 6.9 TB/s, the scaling at 6.0.
// Sums: fp32 over the 64 bytes a thread holds of one chunk, which go into a compensated
// fp32 pair per thread; fp64 across threads and CTAs, always in the same order, so a norm is
// the same in every run. Squares of large and of tiny values do not fit fp32: where a thread's sum
// of a chunk's squares leaves [2^-100, 2^100] it is formed again from scaled values (read from L1) and
// added up in fp64, so that the 2-norm is right for all values of the types (200M fp32 of 1e-3 152 us,
// of 1e-20 166 us; with fp64 squares in place of scaled ones 1483). Between these borders, squares lost
// below fp32's numbers are under 2^-44 of the sum, and a thread's sum over its chunks (2^21 at most)
// stays below 2^121.
// Every CTA of the scaling launch adds up the CTAs' partial sums itself (a few KB from L2), which
// saves a launch in between. The scaling runs through the chunks backwards: the end of the list, which
// the norm has just read, is still in L2.
#include "lce_internal.h"

namespace lce {

namespace {

constexpr int CLIP_THREADS = 512;
constexpr int CLIP_VECS = 4;                                   // 16-byte vectors per thread and chunk
constexpr int CLIP_CHUNK = CLIP_THREADS * CLIP_VECS * 16;      // 32 KB
constexpr int CLIP_CTAS_PER_SM = 4;    // 2048 threads: 128 KB of loads in flight per SM

// A tensor's values seen as the 16-byte vectors of the 128-byte lines that hold them (a warp
// reads whole lines): vectors at both ends may be partly or wholly outside.
struct ClipSpan {
    const uint8_t *base;   // 128-byte aligned, at or before the first value
    uint8_t *out;          // what `base` corresponds to in the destination
    long long lo, hi;      // bytes from base: first value, end
    int dtype;
    bool vec_out;          // the destination has the same alignment
};

template <int CAP> __device__ __forceinline__ ClipSpan clip_span(const ClipTable<CAP> &tb, int i) {
    ClipSpan s;
    const uintptr_t a = reinterpret_cast<uintptr_t>(tb.src[i]);
    const uintptr_t b = reinterpret_cast<uintptr_t>(tb.dst[i]);
    const int off = static_cast<int>(a & 127u);
    s.dtype = static_cast<int>(tb.count[i] & 3);
    s.base = reinterpret_cast<const uint8_t *>(a - off);
    s.out = reinterpret_cast<uint8_t *>(b - off);
    s.lo = off;
    s.hi = off + (tb.count[i] >> 2) * (s.dtype == CE_FP32 ? 4 : 2);
    s.vec_out = ((a ^ b) & 15u) == 0;
    return s;
}

// The tensor that holds chunk c.
template <int CAP> __device__ __forceinline__ int clip_find(const ClipTable<CAP> &tb, int c) {
    int lo = 0, hi = tb.n - 1;   // first[lo] <= c < first[hi + 1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tb.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Reads the vector at byte offset `o`; bytes outside the tensor are zero. LAST: no one
// reads it again.
template <bool LAST> __device__ __forceinline__ uint4 clip_load(const ClipSpan &s, long long o) {
    if (o >= s.lo && o + 16 <= s.hi) {
        const uint4 *a = reinterpret_cast<const uint4 *>(s.base + o);
        return LAST ? __ldcs(a) : *a;
    }
    if (o >= s.hi || o + 16 <= s.lo) return make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (s.dtype == CE_FP32) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (o + 4 * q >= s.lo && o + 4 * q < s.hi)
                w[q] = *reinterpret_cast<const uint32_t *>(s.base + o + 4 * q);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (o + 2 * q >= s.lo && o + 2 * q < s.hi)
                w[q >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(s.base + o + 2 * q))
                             << (16 * (q & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void clip_store(const ClipSpan &s, long long o, const uint4 &v) {
    if (o >= s.lo && o + 16 <= s.hi && s.vec_out) {
        __stcs(reinterpret_cast<uint4 *>(s.out + o), v);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (s.dtype == CE_FP32) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (o + 4 * q >= s.lo && o + 4 * q < s.hi)
                *reinterpret_cast<uint32_t *>(s.out + o + 4 * q) = w[q];
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (o + 2 * q >= s.lo && o + 2 * q < s.hi)
                *reinterpret_cast<uint16_t *>(s.out + o + 2 * q) =
                    static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
    }
}

// The 4 (fp32) or 8 values of a vector.
__device__ __forceinline__ int clip_unpack(const uint4 &v, int dtype, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (dtype == CE_FP32) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[q] = __uint_as_float(w[q]);
            x[q + 4] = 0.f;
        }
        return 4;
    }
    if (dtype == CE_BF16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[2 * q] = __uint_as_float(w[q] << 16);
            x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[q]));
            x[2 * q] = f.x;
            x[2 * q + 1] = f.y;
        }
    }
    return 8;
}
__device__ __forceinline__ uint4 clip_scale(const uint4 &v, int dtype, float f) {
    float x[8];
    clip_unpack(v, dtype, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] *= f;
    uint32_t w[4];
    if (dtype == CE_FP32) {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __float_as_uint(x[q]);
    } else if (dtype == CE_BF16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
            w[q] = *reinterpret_cast<const uint32_t *>(&h);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __half2 h = __floats2half2_rn(x[2 * q], x[2 * q + 1]);
            w[q] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest |g| is found on the bit patterns, whose order is that of the values with
// NaN above infinity: a NaN anywhere is the result.
__device__ __forceinline__ uint32_t clip_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Sum over the block, fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double *red) {
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (l == 0) red[w] = v;
    __syncthreads();
    v = l < CLIP_THREADS / 32 ? red[l] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *red) {
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    v = __reduce_max_sync(0xffffffffu, v);
    if (l == 0) red[w] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, l < CLIP_THREADS / 32 ? red[l] : 0u);
}

// Sums of a thread's squares outside these are formed again from values times 2^-80 or 2^80.
constexpr float CLIP_SQ_MIN = 0x1p-100f, CLIP_SQ_MAX = 0x1p100f;

// The thread's squares of a chunk, `large` or small. Large: the largest value is at least 2^47, and
// 2^48 at most after scaling, so what is lost is below 2^-83 of the sum. Small: values below 2^-50 are below
// 2^30 after scaling, and the square of the smallest, 2^-149, is 2^-138.
__device__ __forceinline__ double clip_squares(const ClipSpan &s, long long o, bool large) {
    const float f = large ? 0x1p-80f : 0x1p80f;
    float a = 0.f, b = 0.f;
#pragma unroll 1
    for (int q = 0; q < CLIP_VECS; ++q) {
        float x[8];
        clip_unpack(clip_load<false>(s, o + q * CLIP_THREADS * 16), s.dtype, x);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            a = fmaf(x[j] * f, x[j] * f, a);
            b = fmaf(x[j + 1] * f, x[j + 1] * f, b);
        }
    }
    return static_cast<double>(a + b) * (large ? 0x1p160 : 0x1p-160);
}

// Adds v to the pair (s, c): s + c is the sum to about twice fp32's precision.
__device__ __forceinline__ void add_pair(float &s, float &c, float v) {
    const float n = s + v;
    const float b = n - s;
    c += (s - (n - b)) + (v - b);
    s = n;
}

template <int CAP>
__global__ void __launch_bounds__(CLIP_THREADS, CLIP_CTAS_PER_SM)
    lce_grad_norm_kernel(const __grid_constant__ ClipTable<CAP> tb, const int kind, double *part) {
    __shared__ double red[CLIP_THREADS / 32];
    __shared__ uint32_t redm[CLIP_THREADS / 32];
    __shared__ double wide[CLIP_THREADS];   // a thread's squares that did not fit fp32
    const int total = tb.first[tb.n];
    wide[threadIdx.x] = 0.0;
    float s = 0.f, c = 0.f;
    uint32_t mx = 0u;
    int i = clip_find(tb, blockIdx.x);
    ClipSpan sp = clip_span(tb, i);
    for (int ch = blockIdx.x; ch < total; ch += gridDim.x) {
        if (ch >= tb.first[i + 1]) {
            while (ch >= tb.first[i + 1]) ++i;
            sp = clip_span(tb, i);
        }
        const long long o = static_cast<long long>(ch - tb.first[i]) * CLIP_CHUNK + threadIdx.x * 16;
        uint4 v[CLIP_VECS];
#pragma unroll
        for (int q = 0; q < CLIP_VECS; ++q) v[q] = clip_load<false>(sp, o + q * CLIP_THREADS * 16);
        float a = 0.f, b = 0.f;
        uint32_t any = 0u;
#pragma unroll
        for (int q = 0; q < CLIP_VECS; ++q) {
            any |= v[q].x | v[q].y | v[q].z | v[q].w;
            float x[8];
            clip_unpack(v[q], sp.dtype, x);
            if (kind == CLIP_NORM_2) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    a = fmaf(x[j], x[j], a);
                    b = fmaf(x[j + 1], x[j + 1], b);
                }
            } else if (kind == CLIP_NORM_1) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    a += fabsf(x[j]);
                    b += fabsf(x[j + 1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) mx = max(mx, clip_bits(x[j]));
            }
        }
        if (kind == CLIP_NORM_2 && !(a + b >= CLIP_SQ_MIN && a + b <= CLIP_SQ_MAX)) {
            if (any & (sp.dtype == CE_FP32 ? 0x7fffffffu : 0x7fff7fffu))
                wide[threadIdx.x] += clip_squares(sp, o, !(a + b < CLIP_SQ_MIN));
            continue;
        }
        add_pair(s, c, a + b);
    }
    if (kind == CLIP_NORM_INF) {
        mx = block_max(mx, redm);
        if (threadIdx.x == 0) part[blockIdx.x] = static_cast<double>(__uint_as_float(mx));
    } else {
        // (an infinite sum has no correction)
        const double v = static_cast<double>(s) + (fabsf(s) < INFINITY ? static_cast<double>(c) : 0.0) +
                         wide[threadIdx.x];
        const double sum = block_sum(v, red);
        if (threadIdx.x == 0) part[blockIdx.x] = sum;
    }
}

// Adds up the partial sums, and scales (tb.n > 0) where the factor is not 1 or `copy`
// says that the destination is another place. One CTA of one launch per call (`tell`)
// writes the norm.
template <int CAP>
__global__ void __launch_bounds__(CLIP_THREADS)
    lce_grad_scale_kernel(const __grid_constant__ ClipTable<CAP> tb, const int kind,
                          const double *part, const int nparts, const float max_norm,
                          const float eps, const int copy, const int tell, float *norm_out) {
    __shared__ double red[CLIP_THREADS / 32];
    __shared__ uint32_t redm[CLIP_THREADS / 32];
    float norm;
    if (kind == CLIP_NORM_INF) {
        uint32_t mx = 0u;
        for (int k = threadIdx.x; k < nparts; k += CLIP_THREADS)
            mx = max(mx, clip_bits(static_cast<float>(part[k])));
        norm = __uint_as_float(block_max(mx, redm));
    } else {
        double v = 0.0;
        for (int k = threadIdx.x; k < nparts; k += CLIP_THREADS) v += part[k];
        v = block_sum(v, red);
        norm = static_cast<float>(kind == CLIP_NORM_2 ? sqrt(v) : v);
    }
    if (tell && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    if (tb.n == 0) return;
    const float f0 = max_norm / (norm + eps);
    const float f = f0 > 1.f ? 1.f : f0;   // NaN stays NaN
    if (f == 1.f && !copy) return;

    const int total = tb.first[tb.n];
    int i = clip_find(tb, total - 1 - static_cast<int>(blockIdx.x));
    ClipSpan sp = clip_span(tb, i);
    for (int ch = total - 1 - static_cast<int>(blockIdx.x); ch >= 0; ch -= gridDim.x) {
        if (ch < tb.first[i]) {
            while (ch < tb.first[i]) --i;
            sp = clip_span(tb, i);
        }
        const long long o = static_cast<long long>(ch - tb.first[i]) * CLIP_CHUNK + threadIdx.x * 16;
        uint4 v[CLIP_VECS];
#pragma unroll
        for (int q = 0; q < CLIP_VECS; ++q) v[q] = clip_load<true>(sp, o + q * CLIP_THREADS * 16);
#pragma unroll
        for (int q = 0; q < CLIP_VECS; ++q) clip_store(sp, o + q * CLIP_THREADS * 16, clip_scale(v[q], sp.dtype, f));
    }
}

template <int CAP>
void fill_table(ClipTable<CAP> &tb, const ClipItem *items, int n) {
    tb.n = n;
    int at = 0;
    for (int i = 0; i < n; ++i) {
        tb.src[i] = items[i].src;
        tb.dst[i] = items[i].dst;
        tb.count[i] = items[i].n * 4 + items[i].dtype;
        tb.first[i] = at;
        at += static_cast<int>(items[i].chunks);
    }
    tb.first[n] = at;
}

int clip_grid(const ClipItem *items, int n, int sms) {
    long long total = 0;
    for (int i = 0; i < n; ++i) total += items[i].chunks;
    long long most = static_cast<long long>(sms) * CLIP_CTAS_PER_SM;
    if (most > CLIP_MAX_PARTS) most = CLIP_MAX_PARTS;
    return static_cast<int>(total < most ? total : most);
}

template <int CAP>
cudaError_t norm_launch(const ClipItem *items, int n, int kind, double *part, int grid, cudaStream_t s) {
    ClipTable<CAP> tb;
    fill_table(tb, items, n);
    lce_grad_norm_kernel<CAP><<<grid, CLIP_THREADS, 0, s>>>(tb, kind, part);
    return cudaGetLastError();
}

template <int CAP>
cudaError_t scale_launch(const ClipItem *items, int n, const ClipScale &c, int grid, cudaStream_t s) {
    ClipTable<CAP> tb;
    fill_table(tb, items, n);
    lce_grad_scale_kernel<CAP><<<grid, CLIP_THREADS, 0, s>>>(tb, c.kind, c.part, c.nparts, c.max_norm, c.eps,
                                                             c.copy, c.tell, c.norm_out);
    return cudaGetLastError();
}

}  // namespace

// Chunks of a tensor of n values at address p.
long long clip_chunks(const void *p, long long n, int dtype) {
    const long long off = static_cast<long long>(reinterpret_cast<uintptr_t>(p) & 127u);
    const long long bytes = off + n * (dtype == CE_FP32 ? 4 : 2);
    return (bytes + CLIP_CHUNK - 1) / CLIP_CHUNK;
}

cudaError_t launch_grad_norm(const ClipItem *items, int n, int kind, double *part, int sms, int *parts,
                             cudaStream_t s) {
    const int grid = clip_grid(items, n, sms);
    *parts = grid;
    if (grid <= 0) return cudaSuccess;
    return n <= CLIP_FEW_TENSORS ? norm_launch<CLIP_FEW_TENSORS>(items, n, kind, part, grid, s)
                                 : norm_launch<CLIP_MAX_TENSORS>(items, n, kind, part, grid, s);
}

cudaError_t launch_grad_scale(const ClipItem *items, int n, const ClipScale &c, int sms, cudaStream_t s) {
    int grid = clip_grid(items, n, sms);
    if (grid < 1) grid = 1;   // the norm alone
    return n <= CLIP_FEW_TENSORS ? scale_launch<CLIP_FEW_TENSORS>(items, n, c, grid, s)
                                 : scale_launch<CLIP_MAX_TENSORS>(items, n, c, grid, s);
}

}  // namespace lce
