// Linear layers with 4-bit weights: out[m][v] = sum over groups g of s[v][g] * sum_{k in g} x[m][k] (q[v][k] - 8),
// q two values a byte (the even one in the low half), s 16-bit, one per row and group of 32, 64 or 128 values.
#include <type_traits>

#include <cuda_fp16.h>

#include "lce_internal.h"
#include "lce_ptx.cuh"

namespace lce {

namespace {

// ------------------------------------------------------------------ few tokens
// Up to 16 tokens per CTA. Bound by reading the weight, so everything else has to fit into the
// time of its bytes: at the measured copy rate an SM gets 23 bytes, 47 weights, a cycle.
//   * A warp takes 16 rows x 128 values (a unit) at a time as the A operand of eight m16n8k16 products, the
//     tokens are the columns of B. Which of the unit's values a product calls its k-th does not
//     matter as long as both operands agree, so a lane's 16 loaded bytes become its fragments as
//     they lie: (w >> n) & mask | magic turns nibbles i and i + 4 of a word into two 16-bit floats
//     16 + q (the nibble lies in the top bits of the mantissa).
//   * The 24 too many of 16 + q go into the accumulator's start, -24 * (sum of the group's x).
//   * Groups of 64 and 32 values need products that stay inside a group: the four lanes of a row exchange
//     words (2 or 4 shuffles a row) so that every product's k lie in one group.
//   * Sums of a group are scaled in fp32 registers and added up over the groups.
//   * KS warps share a row block's units, RG row blocks go on beside each other; what a warp
//     reads next is under way four units ahead, over the ends of row blocks too.
// x lies in shared memory in the order in which lanes take it (one 16-byte load per word).

constexpr int I4_THREADS = 512;
constexpr int I4_WARPS = I4_THREADS / 32;
constexpr int I4_AHEAD = 4;          // units under way per warp
constexpr int I4_UNIT = 128;         // values of k

__device__ __forceinline__ uint32_t lop_and_or(uint32_t a, uint32_t mask, uint32_t bits) { return (a & mask) | bits; }

// 16 + q of nibbles i and i + 4, for i = 0 .. 3.
template <typename T> __device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&o)[4]);
template <> __device__ __forceinline__ void nibbles<__nv_bfloat16>(uint32_t w, uint32_t (&o)[4]) {
    o[0] = lop_and_or(w << 3, 0x00780078u, 0x41804180u);
    o[1] = lop_and_or(w >> 1, 0x00780078u, 0x41804180u);
    o[2] = lop_and_or(w >> 5, 0x00780078u, 0x41804180u);
    o[3] = lop_and_or(w >> 9, 0x00780078u, 0x41804180u);
}
template <> __device__ __forceinline__ void nibbles<__half>(uint32_t w, uint32_t (&o)[4]) {
    o[0] = lop_and_or(w << 6, 0x03c003c0u, 0x4c004c00u);
    o[1] = lop_and_or(w << 2, 0x03c003c0u, 0x4c004c00u);
    o[2] = lop_and_or(w >> 2, 0x03c003c0u, 0x4c004c00u);
    o[3] = lop_and_or(w >> 6, 0x03c003c0u, 0x4c004c00u);
}
constexpr float I4_BIAS = 24.f;   // 16 + q = (q - 8) + 24

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename T> __device__ __forceinline__ float to_float(T v) { return static_cast<float>(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// Word j of lane t (of the four that share a row) is word `w` of chunk `c` of 32 values.
template <int GROUP> __device__ __forceinline__ void word_at(int t, int j, int *c, int *w) {
    if (GROUP == 128) {
        *c = t;
        *w = j;
    } else if (GROUP == 64) {
        *c = (t & 1) + (j & 2);
        *w = (j & 1) + (t & 2);
    } else {
        *c = j;
        *w = t;
    }
}
// The four lanes' words (lane t loaded chunk t) brought into that order.
template <int GROUP> __device__ __forceinline__ void exchange(uint32_t (&u)[4], int t) {
    if constexpr (GROUP != 128) {
        // lanes t and t ^ 2: words 2, 3 of the lower lane against words 0, 1 of the upper one
        const bool up = t & 2;
        const uint32_t s0 = up ? u[0] : u[2], s1 = up ? u[1] : u[3];
        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 2), r1 = __shfl_xor_sync(0xffffffffu, s1, 2);
        if (up) {
            u[0] = r0;
            u[1] = r1;
        } else {
            u[2] = r0;
            u[3] = r1;
        }
        if constexpr (GROUP == 32) {
            // lanes t and t ^ 1: word 1 (3) of the lower lane against word 0 (2) of the upper one
            const bool odd = t & 1;
            const uint32_t a0 = odd ? u[0] : u[1], a1 = odd ? u[2] : u[3];
            const uint32_t b0 = __shfl_xor_sync(0xffffffffu, a0, 1), b1 = __shfl_xor_sync(0xffffffffu, a1, 1);
            if (odd) {
                u[0] = b0;
                u[2] = b1;
            } else {
                u[1] = b0;
                u[3] = b1;
            }
        }
    }
}

// What a warp holds of one unit: 16 bytes of rows r and r + 8, and those rows' scales.
template <int GROUP> struct Unit {
    uint4 q[2];
    uint16_t s[2][I4_UNIT / GROUP];
};

template <typename T, int GROUP, int NT>
__global__ void __launch_bounds__(I4_THREADS, 1) lce_int4_few_kernel(const Int4Params p) {
    constexpr int PER = I4_UNIT / GROUP;     // groups of a unit
    constexpr int JS = 4 / PER;              // words of a lane per group
    extern __shared__ __align__(16) uint8_t i4_smem[];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, tl = lane & 3;
    const int m0 = blockIdx.y * p.tokens;
    const int mt = p.M - m0 < p.tokens ? p.M - m0 : p.tokens;
    const int units = p.units;
    // x as 16-byte pieces [unit][word][token][t], sums of x [group][8 NT] (times -24), partial sums of warps
    uint4 *xw = reinterpret_cast<uint4 *>(i4_smem);
    float *xs = reinterpret_cast<float *>(i4_smem + static_cast<size_t>(units) * 16 * p.tokens * 16);
    float4 *part = reinterpret_cast<float4 *>(xs + static_cast<size_t>(units) * PER * 8 * NT);

    const int ks = p.ks, rg_count = I4_WARPS / ks;
    const int rg = warp / ks, kw = warp % ks;
    const int blocks = (p.V + 15) / 16;
    const int step = gridDim.x * rg_count;
    const int row_bytes = (p.D + 31) / 32 * 16;
    const uint16_t *scale = static_cast<const uint16_t *>(p.scale);
    const int groups = (p.D + GROUP - 1) / GROUP;

    // the warp's sequence of (row block, unit): where the next load goes
    int lb = blockIdx.x * rg_count + rg, lu = kw;
    Unit<GROUP> ring[I4_AHEAD];
    auto fetch = [&](Unit<GROUP> &o) {
        if (lb >= blocks) return;
        const int at = lu * 64 + tl * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = lb * 16 + g + 8 * h < p.V ? lb * 16 + g + 8 * h : p.V - 1;
            o.q[h] = at < row_bytes
                         ? __ldcs(reinterpret_cast<const uint4 *>(p.q + static_cast<long long>(row) * p.ldq + at))
                         : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                o.s[h][i] = lu * PER + i < groups ? scale[static_cast<long long>(row) * p.lds + lu * PER + i]
                                                  : static_cast<uint16_t>(0);
        }
        lu += ks;
        if (lu >= units) {
            lu = kw;
            lb += step;
        }
    };
#pragma unroll
    for (int i = 0; i < I4_AHEAD; ++i) fetch(ring[i]);

    // x into shared memory, beside the first loads
    const T *X = static_cast<const T *>(p.X) + static_cast<long long>(m0) * p.ldx;
    for (int i = t; i < units * 16 * mt; i += I4_THREADS) {
        const int tt = i & 3, m = (i >> 2) % mt, uj = (i >> 2) / mt, j = uj & 3, u = uj >> 2;
        int c, w;
        word_at<GROUP>(tt, j, &c, &w);
        const int k0 = u * I4_UNIT + c * 32 + w * 8;
        const T *src = X + static_cast<long long>(m) * p.ldx + k0;
        uint16_t v[8];
        if (p.x_vec && k0 + 8 <= p.D) {
            const uint4 q = *reinterpret_cast<const uint4 *>(src);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = static_cast<uint16_t>((&q.x)[e / 2] >> (16 * (e & 1)));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = k0 + e < p.D ? reinterpret_cast<const uint16_t *>(src)[e] : static_cast<uint16_t>(0);
        }
        // pairs (0, 4), (1, 5), (2, 6), (3, 7): the order in which a word's nibbles come
        xw[((u * 4 + j) * p.tokens + m) * 4 + tt] =
            make_uint4(v[0] | (v[4] << 16), v[1] | (v[5] << 16), v[2] | (v[6] << 16), v[3] | (v[7] << 16));
    }
    __syncthreads();
    for (int i = t; i < units * PER * 8 * NT; i += I4_THREADS) {
        const int m = i % (8 * NT), gr = i / (8 * NT), u = gr / PER, j0 = gr % PER * JS;
        float s = 0.f;
        if (m < mt)
            for (int j = 0; j < JS; ++j)
                for (int e = 0; e < 4; ++e) {
                    const uint4 q = xw[((u * 4 + j0 + j) * p.tokens + m) * 4 + e];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t w = (&q.x)[h];
                        T lo, hi;
                        *reinterpret_cast<uint16_t *>(&lo) = static_cast<uint16_t>(w);
                        *reinterpret_cast<uint16_t *>(&hi) = static_cast<uint16_t>(w >> 16);
                        s += to_float(lo) + to_float(hi);
                    }
                }
        xs[i] = -I4_BIAS * s;
    }
    __syncthreads();

    float acc[NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    };
    clear();
    auto compute = [&](const Unit<GROUP> &o, int u) {
        uint32_t q0[4] = {o.q[0].x, o.q[0].y, o.q[0].z, o.q[0].w}, q1[4] = {o.q[1].x, o.q[1].y, o.q[1].z, o.q[1].w};
        exchange<GROUP>(q0, tl);
        exchange<GROUP>(q1, tl);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float c[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 b = *reinterpret_cast<const float2 *>(xs + (u * PER + i) * 8 * NT + n * 8 + 2 * tl);
                c[n][0] = c[n][2] = b.x;
                c[n][1] = c[n][3] = b.y;
            }
#pragma unroll
            for (int j = i * JS; j < (i + 1) * JS; ++j) {
                uint32_t a[4], b[4];
                nibbles<T>(q0[j], a);
                nibbles<T>(q1[j], b);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (g + 8 * n < mt) x = xw[((u * 4 + j) * p.tokens + g + 8 * n) * 4 + tl];
                    mma16816<T>(c[n], a[0], b[0], a[1], b[1], x.x, x.y);
                    mma16816<T>(c[n], a[2], b[2], a[3], b[3], x.z, x.w);
                }
            }
            T h0, h1;
            *reinterpret_cast<uint16_t *>(&h0) = o.s[0][i];
            *reinterpret_cast<uint16_t *>(&h1) = o.s[1][i];
            const float s0 = to_float(h0), s1 = to_float(h1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
            }
        }
    };
    // The KS warps' sums of a row block added up by one of them (each in its turn) and written. Two sets of
    // places: a warp that is a row block ahead writes into the other.
    int turn = 0;
    T *out = static_cast<T *>(p.out);
    auto finish = [&](int rb) {
        if (ks > 1) {
            float4 *mine = part + ((turn & 1) * I4_WARPS + warp) * 32 * NT;
#pragma unroll
            for (int n = 0; n < NT; ++n) mine[n * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
            named_bar_sync(1 + rg, ks * 32);
        }
        if (ks == 1 || turn % ks == kw) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float4 s = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                if (ks > 1) {
                    const float4 *from = part + ((turn & 1) * I4_WARPS + rg * ks) * 32 * NT + n * 32 + lane;
                    s = from[0];
                    for (int k = 1; k < ks; ++k) {
                        const float4 o = from[k * 32 * NT];
                        s.x += o.x;
                        s.y += o.y;
                        s.z += o.z;
                        s.w += o.w;
                    }
                }
                const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = n * 8 + 2 * tl + (i & 1), row = rb * 16 + g + 8 * (i >> 1);
                    if (m < mt && row < p.V) out[static_cast<long long>(m0 + m) * p.ldc + row] = from_float<T>(v[i]);
                }
            }
        }
        ++turn;
        clear();
    };
    int cb = blockIdx.x * rg_count + rg, cu = kw;   // (every warp has units: ks is at most a quarter of them)
    while (cb < blocks) {
#pragma unroll
        for (int i = 0; i < I4_AHEAD; ++i) {
            if (cb < blocks) {
                compute(ring[i], cu);
                fetch(ring[i]);
                cu += ks;
                if (cu >= units) {
                    finish(cb);
                    cu = kw;
                    cb += step;
                }
            }
        }
    }
}

// ------------------------------------------------------------------ quantisation
// A warp per row and 256 values: a lane's eight values, the maximum over the lanes of a group.

constexpr int I4Q_THREADS = 256;

template <typename W, typename S>
__global__ void __launch_bounds__(I4Q_THREADS) lce_int4_quantize_kernel(const Int4QuantParams p) {
    const int lane = threadIdx.x & 31;
    const long long task = blockIdx.x * static_cast<long long>(I4Q_THREADS / 32) + (threadIdx.x >> 5);
    const int parts = (p.D + 255) / 256;
    const long long row = task / parts;
    if (row >= p.V) return;
    const int k0 = static_cast<int>(task % parts) * 256 + lane * 8;
    const W *src = static_cast<const W *>(p.W) + row * p.ldw + k0;
    float v[8];
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = k0 + i < p.D ? to_float(src[i]) : 0.f;
        amax = fmaxf(amax, fabsf(v[i]));
        bad |= !(fabsf(v[i]) < INFINITY);
    }
    int any = bad;
    for (int o = p.group / 16; o > 0; o >>= 1) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        any |= __shfl_xor_sync(0xffffffffu, any, o);
    }
    // a seventh of the largest magnitude, as the scale's type has it; a group that holds an infinity or a
    // NaN gets a NaN
    const S s16 = from_float<S>(amax / 7.f);
    float s = to_float(s16);
    if (!(s > 0.f)) s = 1.f;
    if (k0 < (p.D + 31) / 32 * 32) {
        uint32_t q = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = fminf(fmaxf(rintf(v[i] / s), -8.f), 7.f);
            q |= static_cast<uint32_t>(static_cast<int>(r) + 8) << (4 * i);
        }
        *reinterpret_cast<uint32_t *>(p.q + row * p.ldq + k0 / 2) = q;
    }
    if (k0 % p.group == 0 && k0 < p.D)
        static_cast<S *>(p.scale)[row * p.lds + k0 / p.group] = from_float<S>(any ? NAN : s);
}

template <typename T, int GROUP> cudaError_t launch_few(const Int4Params &p, int nt, dim3 grid, size_t smem, cudaStream_t s) {
    if (nt == 1) lce_int4_few_kernel<T, GROUP, 1><<<grid, I4_THREADS, smem, s>>>(p);
    else lce_int4_few_kernel<T, GROUP, 2><<<grid, I4_THREADS, smem, s>>>(p);
    return cudaGetLastError();
}
template <typename T> cudaError_t launch_few_of(const Int4Params &p, int nt, dim3 grid, size_t smem, cudaStream_t s) {
    return p.group == 128 ? launch_few<T, 128>(p, nt, grid, smem, s)
           : p.group == 64 ? launch_few<T, 64>(p, nt, grid, smem, s) : launch_few<T, 32>(p, nt, grid, smem, s);
}

constexpr int I4_MAX_SMEM = 220 * 1024;

size_t few_smem(const Int4Params &p, int tokens, int nt) {
    return static_cast<size_t>(p.units) * (256 * tokens + I4_UNIT / p.group * 32 * nt) + 2 * I4_WARPS * 32 * 16 * nt;
}

template <typename T, int GROUP> cudaError_t set_few() {
    cudaError_t e = cudaFuncSetAttribute(lce_int4_few_kernel<T, GROUP, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         I4_MAX_SMEM);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(lce_int4_few_kernel<T, GROUP, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, I4_MAX_SMEM);
}

template <typename W> cudaError_t launch_quant(const Int4QuantParams &p, cudaStream_t s) {
    const long long tasks = p.V * ((p.D + 255ll) / 256);
    const long long blocks = (tasks + I4Q_THREADS / 32 - 1) / (I4Q_THREADS / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    if (p.scale_dtype == CE_FP16) lce_int4_quantize_kernel<W, __half><<<static_cast<unsigned>(blocks), I4Q_THREADS, 0, s>>>(p);
    else lce_int4_quantize_kernel<W, __nv_bfloat16><<<static_cast<unsigned>(blocks), I4Q_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t int4_set_attributes() {
    cudaError_t e;
    if ((e = set_few<__nv_bfloat16, 128>()) != cudaSuccess) return e;
    if ((e = set_few<__nv_bfloat16, 64>()) != cudaSuccess) return e;
    if ((e = set_few<__nv_bfloat16, 32>()) != cudaSuccess) return e;
    if ((e = set_few<__half, 128>()) != cudaSuccess) return e;
    if ((e = set_few<__half, 64>()) != cudaSuccess) return e;
    return set_few<__half, 32>();
}

cudaError_t launch_int4(Int4Params p, int sms, cudaStream_t s) {
    p.units = (p.D + I4_UNIT - 1) / I4_UNIT;
    // at least four units to a warp, up to eight warps to a row block
    p.ks = 1;
    while (p.ks < 8 && p.units >= 8 * p.ks) p.ks *= 2;
    int tokens = p.M < 16 ? p.M : 16;
    while (tokens > 1 && few_smem(p, tokens, tokens > 8 ? 2 : 1) > I4_MAX_SMEM) --tokens;
    const int nt = tokens > 8 ? 2 : 1;
    p.tokens = tokens;
    const int blocks = (p.V + 15) / 16, per = I4_WARPS / p.ks;
    const int gx = (blocks + per - 1) / per < sms ? (blocks + per - 1) / per : sms;
    const dim3 grid(gx, (p.M + tokens - 1) / tokens);
    const size_t smem = few_smem(p, tokens, nt);
    if (smem > I4_MAX_SMEM) return cudaErrorInvalidValue;
    return p.dtype == CE_FP16 ? launch_few_of<__half>(p, nt, grid, smem, s)
                              : launch_few_of<__nv_bfloat16>(p, nt, grid, smem, s);
}

cudaError_t launch_int4_quantize(const Int4QuantParams &p, cudaStream_t s) {
    return p.dtype == CE_FP32 ? launch_quant<float>(p, s)
           : p.dtype == CE_FP16 ? launch_quant<__half>(p, s) : launch_quant<__nv_bfloat16>(p, s);
}

}  // namespace lce
