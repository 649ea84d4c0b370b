// Linear layers in 8-bit floating point (e4m3) with one fp32 scale per block of 128
// values along the contraction: quantisation, and the product of two such operands.
//
//   rows:  x[r, k] ~ s[r, k / 128] * q[r, k]                 (activations, gradients)
//   tiles: w[n, k] ~ s[n / 128, k / 128] * q[n, k]           (weights)
//   C[m, n] = sum over k blocks b of sa[m, b] * sb[n, b] * sum_{k in b} qa[m, k] qb[n, k]
//
// The scale of a block is the smallest power of two under which its largest finite
// value is at most 448 (e4m3's largest), so the division is exact and e4m3's own rounding
// is the only one; the product takes any fp32 scales.
#include <cstring>
#include <type_traits>

#include <cuda_fp8.h>

#include "lce_internal.h"
#include "lce_ptx.cuh"

namespace lce {

// ------------------------------------------------------------------ quantisation
// One CTA per 128 x 128 tile of X, which its threads hold in registers (8 x 8 values
// each), so X is read once for up to two outputs: row blocks or tiles in X's own layout,
// and the same of X^T (blocks along X's rows), turned through shared memory. Bound by
// HBM bandwidth: 2 (4) bytes read and 1 or 2 written per value. Measured: 4096 x 50256 bf16 in row
// blocks 111 us (5.6 TB/s), X^T 121 us (5.1 TB/s). Rows of 16-bit values that do not start on 16
// bytes come by aligned words: 50257 columns take 158 us (value by value 236; by vectors that lanes
// shift into place between them 242).

namespace {

constexpr int QT_THREADS = 256;

// 2^e of a block whose largest finite |x| is amax, and 2^-e.
struct Pow2 {
    float scale, inv;
};
__device__ __forceinline__ Pow2 block_scale(float amax) {
    const uint32_t b = __float_as_uint(amax);
    // amax = 1.m * 2^x; 448 = 1.75 * 2^8
    int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < -126) e = -126;
    if (b == 0u) e = 0;
    Pow2 s;
    s.scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    s.inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    return s;
}
// e4m3 of a * f and b * f, and of c * f and d * f, in order (f a power of two: exact)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float f) {
    const float2 ff = make_float2(f, f);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(__fmul2_rn(make_float2(a, b), ff), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(__fmul2_rn(make_float2(c, d), ff), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// 8 values of a row as they come (16-bit types stay packed: four words of two), and what the
// kernel needs of them. Maxima ignore NaN; infinities are turned into NaN first (`mend`,
// rarely run), as e4m3 has none.
template <typename T> struct QtVec {
    uint32_t w[4];
    static constexpr uint32_t INF2 = sizeof(T) == 2 && std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
        if constexpr (std::is_same<T, __half>::value) {
            const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
            return *reinterpret_cast<const uint32_t *>(&m);
        } else {
            const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&b));
            return *reinterpret_cast<const uint32_t *>(&m);
        }
    }
    __device__ __forceinline__ static float low(uint32_t v) {
        if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
        else return __uint_as_float(v << 16);
    }
    __device__ __forceinline__ void load(const T *p, int n, bool vec) {
        if (vec && n >= 8) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else if (n >= 8) {
            // a row that starts anywhere: aligned words, of an odd address the first and the last value
            // alone (no byte beside the values is read)
            const uintptr_t a = reinterpret_cast<uintptr_t>(p);
            if (a & 2u) {
                const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
                const uint32_t *u = reinterpret_cast<const uint32_t *>(a + 2);
                const uint32_t first = h[0], last = h[7];
#pragma unroll
                for (int j = 0; j < 3; ++j) w[j] = u[j];
                w[3] = __funnelshift_r(w[2], last, 16);
                w[2] = __funnelshift_r(w[1], w[2], 16);
                w[1] = __funnelshift_r(w[0], w[1], 16);
                w[0] = first | (w[0] << 16);
            } else {
                const uint32_t *u = reinterpret_cast<const uint32_t *>(a);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = u[j];
            }
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (2 * j < n ? h[2 * j] : 0u) | ((2 * j + 1 < n ? static_cast<uint32_t>(h[2 * j + 1]) : 0u) << 16);
        }
    }
    // largest |x| of column pair j, as two 16-bit values
    __device__ __forceinline__ uint32_t abs2(int j) const { return w[j] & 0x7fff7fffu; }
    __device__ __forceinline__ uint32_t row_max() const {
        return max2(max2(abs2(0), abs2(1)), max2(abs2(2), abs2(3)));
    }
    __device__ __forceinline__ void mend() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if ((w[j] & 0x7fffu) == INF2) w[j] |= 0x7fffu;
            if (((w[j] >> 16) & 0x7fffu) == INF2) w[j] |= 0x7fff0000u;
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j >> 1]));
            return j & 1 ? f.y : f.x;
        } else {
            return j & 1 ? __uint_as_float(w[j >> 1] & 0xffff0000u) : __uint_as_float(w[j >> 1] << 16);
        }
    }
};
template <> struct QtVec<float> {
    float x[8];
    __device__ __forceinline__ void load(const float *p, int n, bool vec) {
        if (vec && n >= 8) {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
            const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = j < n ? p[j] : 0.f;
        }
    }
    __device__ __forceinline__ float row_max() const {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
        return m;
    }
    __device__ __forceinline__ void mend() {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (fabsf(x[j]) == INFINITY) x[j] = __uint_as_float(0x7fffffffu);
    }
    __device__ __forceinline__ float get(int j) const { return x[j]; }
};

template <typename T, bool TILE>
__global__ void __launch_bounds__(QT_THREADS, sizeof(T) == 4 ? 2 : 3)
    lce_fp8_quantize_kernel(const Fp8QuantParams p) {
    constexpr bool PACKED = sizeof(T) == 2;
    using V = QtVec<T>;
    __shared__ __align__(16) uint8_t st[128 * 128];
    __shared__ float cred[QT_THREADS / 32][128];
    const int t = threadIdx.x, w = t >> 5, l = t & 31;
    const int i = t & 15, g = t >> 4;          // columns 8 i .. + 7, rows 8 g .. + 7 of the tile
    // (a product launched to overlap may set itself up while this runs; it waits for the end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long tile = blockIdx.x;
    const long long rb = tile / p.cblocks, cb = tile - rb * p.cblocks;
    const long long r0 = rb * 128, c0 = cb * 128;
    const int nr = p.R - r0 < 128 ? static_cast<int>(p.R - r0) : 128;
    const int nc = p.C - c0 < 128 ? static_cast<int>(p.C - c0) : 128;
    const T *X = static_cast<const T *>(p.X) + r0 * p.ld + c0;
    V x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int r = g * 8 + k;
        if (r < nr && i * 8 < nc) x[k].load(X + static_cast<long long>(r) * p.ld + i * 8, nc - i * 8, p.vec != 0);
        else memset(&x[k], 0, sizeof(V));
    }
    // largest |x| of the thread's part of each row
    float rmax[8];
    auto row_maxima = [&]() {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (PACKED) {
                const uint32_t m = x[k].row_max();
                rmax[k] = fmaxf(V::low(m), V::low(m >> 16));
            } else {
                rmax[k] = x[k].row_max();
            }
            rmax[k] = fmaxf(rmax[k], 0.f);   // (a NaN for a thread of NaN only)
        }
    };
    row_maxima();
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) most = fmaxf(most, rmax[k]);
    if (most == INFINITY) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k].mend();
        row_maxima();
        most = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) most = fmaxf(most, rmax[k]);
    }
    Pow2 tile_s = {1.f, 1.f};
    if constexpr (TILE) {
        // (the bit patterns of non-negative floats are in their order)
        const uint32_t mw = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
        if (l == 0) cred[0][w] = __uint_as_float(mw);
        __syncthreads();
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(cred[0][l & 7]));
        tile_s = block_scale(__uint_as_float(m));
        if (t == 0) {
            if (p.q) p.scale[rb * p.cblocks + cb] = tile_s.scale;
            if (p.qt) p.scale_t[cb * p.rblocks + rb] = tile_s.scale;
        }
    }
    if (p.q) {
        if constexpr (!TILE) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) rmax[k] = fmaxf(rmax[k], __shfl_xor_sync(0xffffffffu, rmax[k], o));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = g * 8 + k;
            Pow2 s = tile_s;
            if constexpr (!TILE) {
                s = block_scale(rmax[k]);
                if (i == 0 && r < nr) p.scale[cb * p.R + r0 + r] = s.scale;
            }
            if (r < nr && i * 8 < nc) {
                uint2 v;
                v.x = e4m3x4(x[k].get(0), x[k].get(1), x[k].get(2), x[k].get(3), s.inv);
                v.y = e4m3x4(x[k].get(4), x[k].get(5), x[k].get(6), x[k].get(7), s.inv);
                *reinterpret_cast<uint2 *>(p.q + (r0 + r) * p.ldq + c0 + i * 8) = v;
            }
        }
    }
    if (p.qt) {
        float inv[8];
        if constexpr (TILE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) inv[j] = tile_s.inv;
        } else {
            float m[8];
            if constexpr (PACKED) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t c = x[0].abs2(j);
#pragma unroll
                    for (int k = 1; k < 8; ++k) c = V::max2(c, x[k].abs2(j));
                    c = V::max2(c, __shfl_xor_sync(0xffffffffu, c, 16));
                    m[2 * j] = fmaxf(V::low(c), 0.f);
                    m[2 * j + 1] = fmaxf(V::low(c >> 16), 0.f);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    m[j] = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) m[j] = fmaxf(m[j], fabsf(x[k].get(j)));
                    m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
                }
            }
            if (l < 16) {
                *reinterpret_cast<float4 *>(&cred[w][i * 8]) = make_float4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<float4 *>(&cred[w][i * 8 + 4]) = make_float4(m[4], m[5], m[6], m[7]);
            }
            __syncthreads();
            // thread c: column c's scale, kept in the first row of cred
            if (t < 128) {
                float a = 0.f;
#pragma unroll
                for (int k = 0; k < QT_THREADS / 32; ++k) a = fmaxf(a, cred[k][t]);
                const Pow2 s = block_scale(a);
                cred[0][t] = s.inv;
                if (t < nc) p.scale_t[rb * p.C + c0 + t] = s.scale;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&cred[0][i * 8 + j]);
                inv[j] = v.x; inv[j + 1] = v.y; inv[j + 2] = v.z; inv[j + 3] = v.w;
            }
        }
        // column c's 8-byte unit of rows 8 g .. + 7 goes to unit g ^ (c / 8) of its 128 bytes,
        // which spreads the 16 columns that a half-warp writes at once over all banks
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint2 v;
            v.x = e4m3x4(x[0].get(j), x[1].get(j), x[2].get(j), x[3].get(j), inv[j]);
            v.y = e4m3x4(x[4].get(j), x[5].get(j), x[6].get(j), x[7].get(j), inv[j]);
            *reinterpret_cast<uint2 *>(st + (i * 8 + j) * 128 + ((g ^ i) << 3)) = v;
        }
        __syncthreads();
        const int u = t & 7;   // 16 bytes of a column
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = (t >> 3) + 32 * k;
            const int sw = (c >> 3) & 15;
            uint4 v = *reinterpret_cast<const uint4 *>(st + c * 128 + ((u ^ (sw >> 1)) << 4));
            if (sw & 1) v = make_uint4(v.z, v.w, v.x, v.y);
            if (c < nc && u * 16 < nr) *reinterpret_cast<uint4 *>(p.qt + (c0 + c) * p.ldqt + r0 + u * 16) = v;
        }
    }
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantParams &p, int dtype, bool tile, cudaStream_t s) {
    const long long n = p.rblocks * p.cblocks;
    if (n <= 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>(n);
    if (dtype == CE_FP32) {
        if (tile) lce_fp8_quantize_kernel<float, true><<<grid, QT_THREADS, 0, s>>>(p);
        else lce_fp8_quantize_kernel<float, false><<<grid, QT_THREADS, 0, s>>>(p);
    } else if (dtype == CE_FP16) {
        if (tile) lce_fp8_quantize_kernel<__half, true><<<grid, QT_THREADS, 0, s>>>(p);
        else lce_fp8_quantize_kernel<__half, false><<<grid, QT_THREADS, 0, s>>>(p);
    } else {
        if (tile) lce_fp8_quantize_kernel<__nv_bfloat16, true><<<grid, QT_THREADS, 0, s>>>(p);
        else lce_fp8_quantize_kernel<__nv_bfloat16, false><<<grid, QT_THREADS, 0, s>>>(p);
    }
    return cudaGetLastError();
}

// ------------------------------------------------------------------ product
// tcgen05 kind::f8f6f4 MMAs contract one k block of 128 into a TMEM buffer; the scales
// differ from block to block, so the tile's sum is kept in fp32 registers: as soon as
// a block's partial product is complete, the consumer warps read it from TMEM and add
// sa * sb times it, while the MMAs of the next blocks fill the other buffers.
//
// Roles (384 threads): warps 0-7 consumers (TMEM lane quarter = warp % 4, column half
// = warp / 4), warp 8 TMA producer, warp 9 TMEM owner + MMA issuer, warps 10 and 11 idle
// (registers move between whole warpgroups). A static persistent schedule: unit u of
// cluster c is tile c + u * clusters.
//
// PAIR: a CTA pair per 256 x 256 tile (cta_group::2; each CTA its own 128 rows of A
// and half of B's), for products with many tiles. Otherwise 128 x 128 tiles, one CTA
// each; few tiles are split along k over a cluster of up to 8 CTAs, whose fp32 sums are
// added through distributed shared memory in rank order.
// PARTS: pairs with a long k and few tiles (gradients of an input) take every tile in
// several parts of k, which write fp32 sums into the workspace; lce_fp8_parts_kernel adds them in order.
// Measured with tile scales: 4096 x 8192 x 4096 113 us (2440 TFLOP/s), 4096 x 128256 x 4096 1610 us
// (2680 TFLOP/s; 1700 to 1870 in a row, when the power limit holds the clocks down), 64 x 128256 x 4096 95 us (5.7 TB/s), 1 x 32000 x 4096 28 us (4.7 TB/s; 250 tiles are
// 1.6 per SM). Pairs are bound by the operands' way from L2 into shared memory (32 KB per SM
// and k block in 0.40 us; with a quarter of the MMAs and no reads of TMEM 4096 x 8192 x 4096 takes 89 us),
// then by the handing over of TMEM buffers. Few rows: by HBM.
//
// B_ROWS: B's scales are per row (gradient of a weight); every warp brings those of its
// columns into shared memory of its own. With a whole row of 128 columns per thread, as
// the tiles' path has it, every thread would read all 128 scales per k block: 512 bytes per warp
// and load, 1024 cycles of the shared memory's return path for the CTA. So TMEM is read in the
// layout of matrix fragments: a thread holds 4 rows x 32 columns and reads a quarter of the scales.
// 4096 x 8192 x 4096 takes 183 us, 32000 x 4096 x 2048 389 us: twice the multiplications per value, and
// two warps per scheduler that do not hide one another's latency (149 us without scale loads
// and products; no registers for more columns ahead).
// Every mbarrier wait is bounded, as in the bf16 GEMM. The waits for TMEM buffers acquire at
// CTA scope and their remote arrivals are relaxed: no memory is handed over with them (the
// tcgen05 fences order TMEM), and cluster scope costs a flush or an L1 invalidation per
// k block.

namespace {

constexpr int F8_BK = 128;                 // values (bytes) per k block: one 128-byte swizzle row
constexpr int F8_OP_BYTES = 128 * F8_BK;   // 128 rows of an operand
constexpr int F8_STAGE = 2 * F8_OP_BYTES;  // A and B of one k block, per CTA
constexpr int F8_STAGES = 6;               // pairs; otherwise as many as fit when A has few rows
constexpr int F8_MAX_STAGES = 11;
constexpr int F8_WARP_BOX = 4096;          // 32 rows x 128 bytes of output per consumer warp
constexpr int F8_SMEM = F8_STAGES * F8_STAGE + 8 * F8_WARP_BOX + 1024;
constexpr int F8_THREADS = 384;
// Pairs: a consumer thread holds 128 sums and two TMEM loads of 16 values. 384 threads start
// with 168 registers each; the consumers take 216, the other warpgroup keeps 72:
// 256 * 216 + 128 * 72 = 384 * 168.
constexpr int F8_REGS = 168, F8_REGS_CONSUMER = 216, F8_REGS_OTHER = 72;
static_assert(256 * F8_REGS_CONSUMER + 128 * F8_REGS_OTHER <= F8_THREADS * F8_REGS, "register split");
// Row tiles that run together (they share B in L2): 16384 x 32000 x 4096 takes 1612 us with 16, 1614 with
// 4 or 8 and 1841 with 64; 4096 x 8192 x 4096 114, 118 to 120 and 114.
constexpr int F8_GROUP = 16;

// Instruction descriptor of tcgen05.mma kind::f8f6f4, e4m3 x e4m3 -> fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4)                                // D format: f32
           | (0u << 7) | (0u << 10)                 // A, B format: e4m3
           | (static_cast<uint32_t>(N >> 3) << 17)  // N / 8
           | (static_cast<uint32_t>(M >> 4) << 24); // M / 16
}
template <bool PAIR>
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t f8_cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Tile t: row tiles in groups of F8_GROUP, the rows of a group fastest, then columns.
__device__ __forceinline__ void f8_tile(const Fp8GemmParams &p, int t, int *mt, int *nt) {
    const int per = F8_GROUP * p.n_tiles;
    const int grp = t / per;
    t -= grp * per;
    const int rows = min(F8_GROUP, p.m_tiles - grp * F8_GROUP);
    *nt = t / rows;
    *mt = grp * F8_GROUP + (t - *nt * rows);
}

// 4 columns of the result, of which n exist, at element `at` of C.
__device__ __forceinline__ void f8_store4(void *C, long long at, int n, const float4 &a, int c_type) {
    if (c_type == CE_FP32) {
        const float f[4] = {a.x, a.y, a.z, a.w};
        float *o = static_cast<float *>(C) + at;
        if (n >= 4) *reinterpret_cast<float4 *>(o) = a;
        else
            for (int j = 0; j < n; ++j) o[j] = f[j];
    } else {
        uint16_t *o = static_cast<uint16_t *>(C) + at;
        uint2 u;
        u.x = c_type == CE_FP16 ? pack_f16x2(a.x, a.y) : pack_bf16x2(a.x, a.y);
        u.y = c_type == CE_FP16 ? pack_f16x2(a.z, a.w) : pack_bf16x2(a.z, a.w);
        if (n >= 4) *reinterpret_cast<uint2 *>(o) = u;
        else
            for (int j = 0; j < n; ++j) o[j] = static_cast<uint16_t>((j < 2 ? u.x : u.y) >> (16 * (j & 1)));
    }
}

template <bool PAIR, bool B_ROWS, bool PARTS>
__global__ void __launch_bounds__(F8_THREADS, 1)
    lce_fp8_matmul_kernel(const __grid_constant__ Fp8GemmParams p) {
    constexpr int CL = PAIR ? 2 : 1;
    constexpr int BNT = PAIR ? 256 : 128;
    constexpr int NBUF = TMEM_COLS / BNT;      // partial products in flight
    constexpr int COLS = BNT / 2;              // columns per consumer warp
    static_assert(F8_STAGES >= NBUF, "a stage's phase must outlive its TMEM buffer");
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[F8_MAX_STAGES];
    // the MMAs of a stage have ended: the producer may fill it again, and the consumers may read
    // its TMEM buffer (one commit for both; a stage comes around no sooner than its buffer, which
    // the consumers have released by then, so no phase can be missed)
    __shared__ __align__(8) uint64_t done_bar[F8_MAX_STAGES];
    __shared__ __align__(8) uint64_t tempty_bar[NBUF];
    __shared__ __align__(8) uint64_t drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), csize = f8_cluster_size();
    const uint32_t crank = PAIR ? rank : 0u;
    const bool leader = crank == 0;
    const int cid = static_cast<int>(blockIdx.x / csize), ncl = static_cast<int>(gridDim.x / csize);
    // k blocks of this CTA (of unit t, PARTS): all, or its part of a split product
    auto k_begin = [&](int t) {
        if constexpr (PARTS) return static_cast<int>(static_cast<long long>(p.KB) * (t / p.tiles) / p.parts);
        else return PAIR ? 0 : static_cast<int>(static_cast<long long>(p.KB) * rank / csize);
    };
    auto k_end = [&](int t) {
        if constexpr (PARTS) return static_cast<int>(static_cast<long long>(p.KB) * (t / p.tiles + 1) / p.parts);
        else return PAIR ? p.KB : static_cast<int>(static_cast<long long>(p.KB) * (rank + 1) / csize);
    };
    const int units = PARTS ? p.tiles * p.parts : p.tiles;
    // A single token's A takes 1 KB of a stage, not 16: more stages, more bytes of B under way.
    // (The MMA reads 128 rows of A all the same, the rest of them out of B: rows of no output.)
    const int a_bytes = PAIR ? F8_OP_BYTES : p.a_box_rows * F8_BK;
    const int stage_bytes = PAIR ? F8_STAGE : a_bytes + F8_OP_BYTES;
    const int nstages = PAIR ? F8_STAGES : p.stages;

    if (threadIdx.x == 0) {
        for (int s = 0; s < nstages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&done_bar[s], 1);
        }
        for (int b = 0; b < NBUF; ++b) mbar_init(&tempty_bar[b], CL * NUM_EPI_WARPS);
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == PRODUCER_WARP && lane == 0) {
        prefetch_tmap(&p.tmA);
        prefetch_tmap(&p.tmB);
        if (p.n_bulk > 0) prefetch_tmap(&p.tmC);
    }
    if (warp == MMA_WARP) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&tmem_slot)),
                         "r"(TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&tmem_slot)),
                         "r"(TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();   // the peer's barriers exist from here on
    tc_fence_after();
    const uint32_t tmem_base = tmem_slot;
    // what was launched before has ended (at once, unless its launch was allowed to overlap)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // cleared here, long before the first wait of any CTA can run out
    if (blockIdx.x == 0 && threadIdx.x == 0) *(volatile int *)(p.hdr + HDR_FLAG) = 0;

    Abort ab;
    ab.flag_smem = &abort_flag;
    ab.hdr = p.hdr;
    ab.limit_ns = p.timeout_ns;

    if (warp >= NUM_EPI_WARPS) {
        if constexpr (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F8_REGS_OTHER));
        if (warp == PRODUCER_WARP && lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            const uint32_t bytes = static_cast<uint32_t>(stage_bytes);
            for (int t = cid; ok && t < units; t += ncl) {
                int mt, nt;
                f8_tile(p, PARTS ? t % p.tiles : t, &mt, &nt);
                const int kb0 = k_begin(t), kb1 = k_end(t);
                const int ya = mt * (CL * 128) + static_cast<int>(crank) * 128;
                const int yb = nt * BNT + static_cast<int>(crank) * 128;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&done_bar[stage], phase ^ 1, ab)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sA = smem + stage * stage_bytes;
                    uint8_t *sB = sA + a_bytes;
                    uint64_t *fb = &full_bar[stage];
                    if constexpr (PAIR) {
                        // both CTAs' bytes complete on the leader's barrier
                        if (leader) mbar_arrive_expect_tx(fb, 2 * bytes);
                        const uint32_t lfb = map_to_rank(fb, 0);
                        tma_load_2d_pair(sA, &p.tmA, lfb, kb * F8_BK, ya);
                        tma_load_2d_pair(sB, &p.tmB, lfb, kb * F8_BK, yb);
                    } else {
                        mbar_arrive_expect_tx(fb, bytes);
                        tma_load_2d(sA, &p.tmA, fb, kb * F8_BK, ya);
                        tma_load_2d(sB, &p.tmB, fb, kb * F8_BK, yb);
                    }
                    ++issued;
                    if (++stage == nstages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) {
                // drain: wait (bounded) for the copies still in flight into each stage
                const int n = issued < nstages ? issued : nstages;
                for (int i = 0; i < n; ++i) {
                    if (--stage < 0) {
                        stage = nstages - 1;
                        phase ^= 1;
                    }
                    if (leader) mbar_wait_drain(&full_bar[stage], phase, 50000000ull);
                }
                if (!leader) {
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 50000000ull) {}
                }
            }
        } else if (warp == MMA_WARP && leader) {
            // the whole warp goes along (its loop counters stay in uniform registers, which the
            // MMAs take their operands from); one lane issues
            int stage = 0;
            uint32_t phase = 0;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true, any_mma = false;
            constexpr uint32_t idesc = idesc_e4m3(CL * 128, BNT);
            constexpr uint16_t both = static_cast<uint16_t>((1u << CL) - 1u);
            for (int t = cid; ok && t < units; t += ncl) {
                const int nk = k_end(t) - k_begin(t);
                for (int kb = 0; kb < nk; ++kb) {
                    const uint32_t sA = smem_u32(smem + stage * stage_bytes);
                    const uint64_t ad = sdesc(sA, 16u, 1024u);
                    const uint64_t bd = sdesc(sA + a_bytes, 16u, 1024u);
                    const uint32_t d = tmem_base + buf * BNT;
                    ok = mbar_wait(&full_bar[stage], phase, ab) && mbar_wait(&tempty_bar[buf], bphase ^ 1, ab);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 values (bytes) of k per MMA
                            umma_e4m3<PAIR>(d, ad + static_cast<uint64_t>(k * 2),
                                            bd + static_cast<uint64_t>(k * 2), idesc, k != 0 ? 1u : 0u);
                        if constexpr (PAIR) umma_commit_pair(&done_bar[stage], both);
                        else umma_commit(&done_bar[stage]);
                    }
                    __syncwarp();
                    any_mma = true;
                    if (++stage == nstages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    if (++buf == NBUF) {
                        buf = 0;
                        bphase ^= 1;
                    }
                }
            }
            if (any_mma) {
                // every MMA (and every arrival it sends to the peer) has completed
                // before TMEM is freed and the CTAs leave
                if (elect_one()) {
                    if constexpr (PAIR) umma_commit_pair(&drain_bar, both);
                    else umma_commit(&drain_bar);
                }
                __syncwarp();
                mbar_wait_drain(&drain_bar, 0, 50000000ull);
            }
        }
    } else {
        if constexpr (PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F8_REGS_CONSUMER));
        const int quarter = warp & 3, half = warp >> 2;
        uint8_t *box = smem + F8_STAGES * F8_STAGE + warp * F8_WARP_BOX;
        // B_ROWS: the scales of the warp's columns for two k blocks, in its output box (free
        // between a tile's store and the next one's)
        float *sb_smem = reinterpret_cast<float *>(box);
        const uint32_t tempty_addr = map_to_rank(&tempty_bar[0], PAIR ? 0u : rank);
        int buf = 0, stage = 0;
        uint32_t phase = 0;
        int par = 0;
        bool ok = true;
        for (int t = cid; ok && t < units; t += ncl) {
            int mt, nt;
            f8_tile(p, PARTS ? t % p.tiles : t, &mt, &nt);
            const int kb0 = k_begin(t), kb1 = k_end(t);
            const int row0 = mt * (CL * 128) + static_cast<int>(crank) * 128 + quarter * 32;
            const int col0 = nt * BNT + half * COLS;
            const bool active = row0 < p.M && col0 < p.N;   // warp-uniform: some output of this warp exists
            // each lane brings the scale of one row; a thread's rows are that one or (fragments) four, 8
            // apart, which it gets from the lanes that have them
            constexpr int ROWS = B_ROWS ? 4 : 1;
            const int row = row0 + lane;
            const float *sa = p.sa + static_cast<long long>(row < p.M ? row : 0) * p.sa_row;
            const long long sbk = p.sb_block;
            // tile scales: the warp's columns lie in one block of 128; row scales: VEC columns per lane
            constexpr int VEC = COLS / 32;
            const int sb_col = col0 + lane * VEC;
            const float *sb = p.sb + (B_ROWS ? static_cast<long long>(sb_col < p.N ? sb_col : 0)
                                             : static_cast<long long>(col0 < p.N ? col0 / 128 : 0)) * p.sb_row;
            auto load_sb = [&](float (&b)[VEC], int kb) {
                const float *at = sb + kb * sbk;
                if constexpr (!B_ROWS) {
                    b[0] = *at;
                } else if (p.sb_vec && sb_col + VEC <= p.N) {
                    if constexpr (VEC == 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(at);
                        b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
                    } else {
                        const float2 v = *reinterpret_cast<const float2 *>(at);
                        b[0] = v.x; b[1] = v.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) b[j] = sb_col + j < p.N ? at[j * p.sb_row] : 0.f;
                }
            };
            if constexpr (B_ROWS) {
                if (lane == 0) bulk_wait_read0();
                __syncwarp();
            }
            // scales of the next k block, and (where registers allow) of the one after it
            constexpr int AHEAD = B_ROWS ? 1 : 2;
            float a0, a1 = 0.f, b0[VEC], b1[VEC];
            a0 = sa[kb0 * p.sa_block];
            load_sb(b0, kb0);
            if (AHEAD > 1 && kb0 + 1 < kb1) {
                a1 = sa[(kb0 + 1) * p.sa_block];
                load_sb(b1, kb0 + 1);
            }
            // the thread's sums: columns 2 j and 2 j + 1 of its row, or (fragments) of group g of 8
            // columns and row i: acc[4 g + i]
            float2 acc[COLS / 2];
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j) acc[j] = make_float2(0.f, 0.f);
            for (int kb = kb0; kb < kb1; ++kb) {
                float s[ROWS];
#pragma unroll
                for (int i = 0; i < ROWS; ++i) s[i] = B_ROWS ? __shfl_sync(0xffffffffu, a0, lane / 4 + 8 * i) : a0;
                if constexpr (B_ROWS) {
                    // Columns 2 f + 8 q (+ 1) of 32 belong to the lanes with lane % 4 = f: they are kept side by
                    // side, at 8 f + 2 q. (The other k block's half may still be in use by a slower lane.)
                    float *to = sb_smem + par * COLS + lane * VEC / 32 * 32 + lane * VEC % 32 / 8 * 2;
#pragma unroll
                    for (int j = 0; j < VEC; j += 2)
                        *reinterpret_cast<float2 *>(to + (lane * VEC % 8 / 2 + j / 2) * 8) = make_float2(b0[j], b0[j + 1]);
                    __syncwarp();
                } else {
                    s[0] *= b0[0];
                }
                if constexpr (AHEAD > 1) {
                    a0 = a1;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) b0[j] = b1[j];
                }
                if (kb + AHEAD < kb1) {
                    (AHEAD > 1 ? a1 : a0) = sa[(kb + AHEAD) * p.sa_block];
                    load_sb(AHEAD > 1 ? b1 : b0, kb + AHEAD);
                }
                ok = mbar_wait(&done_bar[stage], phase, ab);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(tempty_addr + buf * 8);
                };
                if (active) {
                    tc_fence_after();
                    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                           static_cast<uint32_t>(buf * BNT + half * COLS);
                    // (each load runs beside the arithmetic on the last one)
                    uint32_t v[2][16];
                    if constexpr (B_ROWS) {
                        // loads: 32 columns of rows 0-15, then of rows 16-31 of the quarter
                        constexpr int LOADS = COLS / 16;
                        float4 bq[2];   // scales of the thread's 8 columns of 32
                        tmem_ldfrag_start(taddr, v[0]);
                        tmem_ld16_wait(v[0]);
#pragma unroll
                        for (int c = 0; c < LOADS; ++c) {
                            if (c % 2 == 0) {
                                const float4 *from =
                                    reinterpret_cast<const float4 *>(sb_smem + par * COLS + c / 2 * 32 + (lane & 3) * 8);
                                bq[0] = from[0];
                                bq[1] = from[1];
                            }
                            if (c + 1 < LOADS)
                                tmem_ldfrag_start(taddr + ((c + 1) / 2) * 32 + ((c + 1) % 2) * (16u << 16), v[(c + 1) & 1]);
                            else
                                release();   // everything is in registers
                            const uint32_t(&u)[16] = v[c & 1];
                            const int i0 = (c % 2) * 2;   // rows i0 and i0 + 1 of the thread
                            const float2 sa0 = make_float2(s[i0], s[i0]), sa1 = make_float2(s[i0 + 1], s[i0 + 1]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int g = (c / 2) * 4 + q;
                                const float2 b = q % 2 ? make_float2(bq[q / 2].z, bq[q / 2].w)
                                                       : make_float2(bq[q / 2].x, bq[q / 2].y);
                                float2 &x = acc[4 * g + i0], &y = acc[4 * g + i0 + 1];
                                x = __ffma2_rn(make_float2(__uint_as_float(u[4 * q]), __uint_as_float(u[4 * q + 1])),
                                               __fmul2_rn(sa0, b), x);
                                y = __ffma2_rn(
                                    make_float2(__uint_as_float(u[4 * q + 2]), __uint_as_float(u[4 * q + 3])),
                                    __fmul2_rn(sa1, b), y);
                            }
                            if (c + 1 < LOADS) tmem_ld16_wait(v[(c + 1) & 1]);
                        }
                    } else {
                        const float2 s2 = make_float2(s[0], s[0]);
                        tmem_ld16_start(taddr, v[0]);
                        tmem_ld16_wait(v[0]);
#pragma unroll
                        for (int c = 0; c < COLS / 16; ++c) {
                            if (c + 1 < COLS / 16) tmem_ld16_start(taddr + (c + 1) * 16, v[(c + 1) & 1]);
                            else release();   // everything is in registers
                            const uint32_t(&u)[16] = v[c & 1];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                acc[c * 8 + j] = __ffma2_rn(
                                    make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])), s2,
                                    acc[c * 8 + j]);
                            if (c + 1 < COLS / 16) tmem_ld16_wait(v[(c + 1) & 1]);
                        }
                    }
                } else {
                    release();
                }
                if (++buf == NBUF) buf = 0;
                if (++stage == nstages) {
                    stage = 0;
                    phase ^= 1;
                }
                par ^= 1;
            }
            if (!ok) break;
            if constexpr (B_ROWS) __syncwarp();   // the scales have been read
            if (!PAIR && csize > 1) {
                // one tile per cluster: the stages are free (all copies landed, all MMAs done); the
                // partial sums as 128 x 128 fp32, 16-byte chunk j of row r at j ^ (r % 8)
                if constexpr (B_ROWS) {
#pragma unroll
                    for (int g = 0; g < COLS / 8; ++g)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = quarter * 32 + lane / 4 + 8 * i, col = half * COLS + g * 8 + (lane & 3) * 2;
                            *reinterpret_cast<float2 *>(reinterpret_cast<float *>(smem) + r * 128 +
                                                        (((col >> 2) ^ (r & 7)) << 2) + (col & 2)) = acc[4 * g + i];
                        }
                } else {
                    const int r = quarter * 32 + lane;
                    float *dst = reinterpret_cast<float *>(smem) + r * 128;
#pragma unroll
                    for (int j = 0; j < COLS / 4; ++j)
                        *reinterpret_cast<float4 *>(dst + (((half * (COLS / 4) + j) ^ (r & 7)) << 2)) =
                            make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
                }
                break;
            }
            if (active) {
                // 128-byte wide boxes of 32 rows: 64 columns of 16 bits, or 32 of fp32
                const int per = p.c_type == CE_FP32 ? 32 : 64;
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    const int bx = col0 + c * 32 / per * per;   // the box's first column
                    if (bx >= p.N) continue;
                    const bool first = c * 32 % per == 0, last = (c * 32 + 32) % per == 0;
                    if (first) {
                        if (lane == 0) bulk_wait_read0();
                        __syncwarp();
                    }
                    if constexpr (B_ROWS) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int r = lane / 4 + 8 * i;
                                const float2 a = acc[c * 16 + 4 * q + i];
                                if (p.c_type == CE_FP32) {
                                    const int j = 2 * q + ((lane & 3) >> 1);
                                    *reinterpret_cast<float2 *>(box + r * 128 + ((j ^ (r & 7)) << 4) + (lane & 1) * 8) = a;
                                } else {
                                    const int j = (c & 1) * 4 + q;
                                    *reinterpret_cast<uint32_t *>(box + r * 128 + ((j ^ (r & 7)) << 4) + (lane & 3) * 4) =
                                        p.c_type == CE_FP16 ? pack_f16x2(a.x, a.y) : pack_bf16x2(a.x, a.y);
                                }
                            }
                    } else if (p.c_type == CE_FP32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4 *>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                                make_float4(acc[c * 16 + 2 * j].x, acc[c * 16 + 2 * j].y,
                                            acc[c * 16 + 2 * j + 1].x, acc[c * 16 + 2 * j + 1].y);
                    } else {
                        const int jb = (c & 1) * 4;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float2 a = acc[c * 16 + 4 * j + q];
                                w[q] = p.c_type == CE_FP16 ? pack_f16x2(a.x, a.y) : pack_bf16x2(a.x, a.y);
                            }
                            *reinterpret_cast<uint4 *>(box + lane * 128 + (((jb + j) ^ (lane & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (last) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && bx < p.n_bulk) {
                            tma_store_2d(&p.tmC, box, bx, PARTS ? row0 + t / p.tiles * (p.m_tiles * 256) : row0);
                            bulk_commit();
                        }
                        // a bulk store writes whole 16-byte pieces of a row: what N leaves in its last
                        // piece is copied value by value
                        if (p.n_bulk < p.N && bx + per > p.n_bulk && row0 + lane < p.M) {
                            const int elem = p.c_type == CE_FP32 ? 4 : 2;
                            for (int col = max(bx, p.n_bulk); col < min(p.N, bx + per); ++col) {
                                const int o = (col - bx) * elem;
                                const uint8_t *from = box + lane * 128 + (((o >> 4) ^ (lane & 7)) << 4) + (o & 15);
                                uint8_t *to = static_cast<uint8_t *>(p.C) + ((row0 + lane) * p.ldc + col) * elem;
                                if (elem == 4) *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(from);
                                else *reinterpret_cast<uint16_t *>(to) = *reinterpret_cast<const uint16_t *>(from);
                            }
                        }
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // no CTA of a pair leaves while the other may still write to it; partial sums are in place
    if (csize > 1) cluster_sync_all();
    if (!PAIR && csize > 1) {
        // rows of this CTA: 128 / csize; a warp adds up one row at a time, 4 columns per lane
        int mt, nt;
        f8_tile(p, cid, &mt, &nt);
        const int rows = 128 / static_cast<int>(csize);
        const int col = nt * BNT + lane * 4;
        for (int k = warp; k < rows && warp < NUM_EPI_WARPS; k += NUM_EPI_WARPS) {
            const int r = static_cast<int>(rank) * rows + k;
            const long long row = static_cast<long long>(mt) * 128 + r;
            if (row >= p.M || col >= p.N) continue;
            const float *src = reinterpret_cast<const float *>(smem) + r * 128 + ((lane ^ (r & 7)) << 2);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t q = 0; q < csize; ++q) {
                const float4 v = ld_cluster_f4(map_to_rank(src, q));
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
            f8_store4(p.C, row * p.ldc + col, p.N - col, a, p.c_type);
        }
        cluster_sync_all();   // no CTA leaves while a peer may still read its partial sums
    }
    if (warp == MMA_WARP) {
        tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(TMEM_COLS)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(TMEM_COLS)
                         : "memory");
    }
}

// Adds the parts of a product: 4 columns per thread. Bound by L2.
constexpr int FP_THREADS = 256;
__global__ void __launch_bounds__(FP_THREADS)
    lce_fp8_parts_kernel(const float *part, const int parts, const long long part_size, const int ld, const int M,
                         const int N, void *C, const long long ldc, const int c_type) {
    const int vecs = ld / 4;
    const long long i = static_cast<long long>(blockIdx.x) * FP_THREADS + threadIdx.x;
    const int row = static_cast<int>(i / vecs), col = static_cast<int>(i % vecs) * 4;
    if (row >= M || col >= N) return;
    const float *src = part + static_cast<long long>(row) * ld + col;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < parts; ++q) {
        const float4 v = *reinterpret_cast<const float4 *>(src + q * part_size);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
    }
    f8_store4(C, row * ldc + col, N - col, a, c_type);
}

using Fp8Kernel = void (*)(const Fp8GemmParams);
Fp8Kernel fp8_kernel(bool pair, bool b_rows, bool parts) {
    if (parts) return lce_fp8_matmul_kernel<true, false, true>;
    if (pair) return b_rows ? lce_fp8_matmul_kernel<true, true, false> : lce_fp8_matmul_kernel<true, false, false>;
    return b_rows ? lce_fp8_matmul_kernel<false, true, false> : lce_fp8_matmul_kernel<false, false, false>;
}

}  // namespace

cudaError_t fp8_set_attributes() {
    for (int k = 0; k < 5; ++k) {
        const bool parts = k == 4;
        const Fp8Kernel f = fp8_kernel(k & 1, k & 2, parts);
        cudaError_t e;
        if ((k & 1) || parts) {
            // the register split waits forever for registers that the launch does not have
            cudaFuncAttributes fa{};
            e = cudaFuncGetAttributes(&fa, f);
            if (e != cudaSuccess) return e;
            if (fa.numRegs < F8_REGS) return cudaErrorInvalidKernelImage;
        }
        e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, F8_SMEM);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_fp8_matmul(const Fp8GemmParams &p, bool pair, bool b_rows, int cluster, int clusters,
                              bool overlap, cudaStream_t s) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster * clusters));
    cfg.blockDim = dim3(F8_THREADS);
    cfg.dynamicSmemBytes = F8_SMEM;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (overlap) {
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, fp8_kernel(pair, b_rows, p.parts > 1), p);
}

cudaError_t launch_fp8_parts(const Fp8GemmParams &p, void *out, long long ldc, int c_type, cudaStream_t s) {
    const long long n = static_cast<long long>(p.M) * (p.ldc / 4);
    lce_fp8_parts_kernel<<<static_cast<unsigned>((n + FP_THREADS - 1) / FP_THREADS), FP_THREADS, 0, s>>>(
        static_cast<const float *>(p.C), p.parts, static_cast<long long>(p.m_tiles) * 256 * p.ldc,
        static_cast<int>(p.ldc), p.M, p.N, out, ldc, c_type);
    return cudaGetLastError();
}

}  // namespace lce
