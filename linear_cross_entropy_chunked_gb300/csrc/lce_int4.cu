// Linear layers with 4-bit weights: out[m][v] = sum over groups g of s[v][g] * sum_{k in g} x[m][k] (q[v][k] - 8),
// q two values a byte (the even one in the low half), s 16-bit, one per row and group of 32, 64 or 128 values.
#include <type_traits>

#include <cuda_fp16.h>

#include "lce_internal.h"
#include "lce_ptx.cuh"

namespace lce {

namespace {

// ------------------------------------------------------------------ few tokens
// Up to 8 tokens. Bound by reading the weight, so everything else has to fit into the
// time of its bytes: at the measured copy rate an SM gets 23 bytes, 47 weights, a cycle.
//   * A warp takes 16 rows x 128 values (a unit) at a time as the A operand of eight m16n8k16 products, the
//     tokens are the columns of B. Which of the unit's values a product calls its k-th does not
//     matter as long as both operands agree, so a lane's 16 loaded bytes become its fragments as
//     they lie: of a word's nibbles i and i + 4, masked into 16-bit floats 1024 + q or 1024 + 16 q, one
//     packed fp16 operation makes q - 8, exactly: 5 operations of the half-rate integer pipe per eight values.
//   * The products are fp16 for bf16 x too (whose 7 bits of mantissa would take 8 such operations): a
//     token is multiplied by the power of two that brings its largest magnitude below 2^15. bf16's
//     8 bits fit; what lies below 2^-29 of the largest is rounded to multiples of 2^-39 of it.
//   * Groups of 64 and 32 values need products that stay inside a group: the four lanes of a row exchange
//     words (2 or 4 shuffles a row) so that every product's k lie in one group.
//   * Sums of a group are scaled in fp32 registers and added up over the groups.
//   * A CTA has a range of row blocks, and of its chunks (16 rows x 4 units) each warp a range of its own, so all
//     warps have the same to do whatever V and D are. Nothing holds them together: each brings its
//     chunks by bulk copies (a row's 256 bytes each) into buffers of its own. A row block that two or
//     more warps have parts of is added up at the end.
// x lies in shared memory in the order in which lanes take it (one 16-byte load per word).

constexpr int I4_UNIT = 128;         // values of k
constexpr int I4_CHUNK = 8;          // units of a chunk
constexpr int I4_RING = 2;           // chunks of a warp: one at hand, two under way
// A chunk in shared memory: its even rows, then, half a line (64 bytes) further on than that, its odd rows:
// the lanes of two rows read different banks.
constexpr int I4_ROW = I4_CHUNK * 64;
constexpr int I4_ODD = 8 * I4_ROW + 64;
constexpr int I4_BUF = 16 * I4_ROW + 128;
constexpr int I4_MAX_WARPS = 16;
constexpr uint64_t I4_WAIT_NS = 2000000000ull;    // bound of a wait for copies (2 s)

// (a & MASK) | bits in one operation: `bits` has to be in a register for that.
template <uint32_t MASK> __device__ __forceinline__ __half2 and_or(uint32_t a, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "n"(MASK), "r"(bits));
    return *reinterpret_cast<const __half2 *>(&r);
}
// q - 8 of nibbles i and i + 4 of a word, for i = 0 .. 3, as pairs of fp16; magic: 0x64006400 (1024, twice).
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t magic, __half2 (&o)[4]) {
    const __half2 sixteenth = __float2half2_rn(0.0625f);
    const __half2 off0 = __float2half2_rn(-1032.f), off1 = __float2half2_rn(-72.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t v = i ? w >> 8 : w;
        o[2 * i] = __hadd2(and_or<0x000f000fu>(v, magic), off0);
        o[2 * i + 1] = __hfma2(and_or<0x00f000f0u>(v, magic), sixteenth, off1);
    }
}
template <int OFF> __device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr), "n"(OFF));
    return v;
}
template <int OFF> __device__ __forceinline__ float lds32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1 + %2];" : "=f"(v) : "r"(addr), "n"(OFF));
    return v;
}

// c (+)= A B; `first`: c starts from zero.
__device__ __forceinline__ void mma16816(float (&c)[4], __half2 a0, __half2 a1, __half2 a2, __half2 a3, uint32_t b0,
                                         uint32_t b1, bool first) {
    if (first) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %10, %10, %10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(*reinterpret_cast<uint32_t *>(&a0)), "r"(*reinterpret_cast<uint32_t *>(&a1)),
                       "r"(*reinterpret_cast<uint32_t *>(&a2)), "r"(*reinterpret_cast<uint32_t *>(&a3)), "r"(b0),
                       "r"(b1), "f"(0.f));
        return;
    }
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(*reinterpret_cast<uint32_t *>(&a0)), "r"(*reinterpret_cast<uint32_t *>(&a1)),
                   "r"(*reinterpret_cast<uint32_t *>(&a2)), "r"(*reinterpret_cast<uint32_t *>(&a3)), "r"(b0), "r"(b1));
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

template <typename T, int GROUP>
__global__ void __launch_bounds__(I4_MAX_WARPS * 32, 1) lce_int4_few_kernel(const Int4Params p) {
    constexpr int PER = I4_UNIT / GROUP;     // groups of a unit
    constexpr int JS = 4 / PER;              // words of a lane per group
    constexpr int SC = I4_CHUNK * PER;       // scales of a chunk's row
    extern __shared__ __align__(128) uint8_t i4_smem[];
    __shared__ float s_up[8], s_down[8];   // a token's power of two, and its inverse
    __shared__ unsigned s_max[8];           // the bits of its largest finite magnitude
    __shared__ __align__(8) uint64_t bars[I4_MAX_WARPS][I4_RING];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, tl = lane & 3;
    const int threads = blockDim.x, warps = threads / 32;
    const int mt = p.M;
    const int units = p.units;
    // per warp: the ring's chunks of the weight, and of scales (fp32 [16][SC]); then 256 bytes of zeros, and x as
    // 16-byte pieces [unit][token][word][t], the words of odd tokens in the order 1 0 3 2 (two tokens' pieces
    // of a word lie half a line apart)
    uint8_t *mine = i4_smem + warp * (I4_RING * I4_BUF);
    float *my_scales = reinterpret_cast<float *>(i4_smem + warps * (I4_RING * I4_BUF)) + warp * (I4_RING * 16 * SC);
    uint4 *zero = reinterpret_cast<uint4 *>(i4_smem + warps * (I4_RING * (I4_BUF + 16 * SC * 4)));
    uint4 *xw = zero + 16;

    const int blocks = (p.V + 15) / 16;
    const int row_bytes = (p.D + 31) / 32 * 16;
    const int groups = (p.D + GROUP - 1) / GROUP;
    // the CTA's row blocks, and the warp's chunks of them
    const int b0 = static_cast<int>(static_cast<long long>(blocks) * blockIdx.x / gridDim.x);
    const int b1 = static_cast<int>(static_cast<long long>(blocks) * (blockIdx.x + 1) / gridDim.x);
    const int cpb = (units + I4_CHUNK - 1) / I4_CHUNK;   // chunks of a row block
    const long long chunks = static_cast<long long>(b1 - b0) * cpb;
    auto begin_of = [&](int w) -> int { return static_cast<int>(chunks * w / warps); };
    const int c_end = begin_of(warp + 1);

    if (t < warps * I4_RING) mbar_init(&bars[t / I4_RING][t % I4_RING], 1);
    if (t < 16) {
        zero[t] = make_uint4(0u, 0u, 0u, 0u);
        if (t < 8) s_max[t] = 0u;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();

    // what is brought next: chunk nc, which is chunk `nk` of row block `nb`; where it lies, for the lane's row (of
    // 16) and scales
    constexpr int NS = (16 * SC + 31) / 32;
    int nc = begin_of(warp), nb = b0 + nc / cpb, nk = nc % cpb;
    const uint8_t *src = nullptr;
    const T *sp[NS];
    float sc[NS];           // the scales that were asked for last
    auto rows_at = [&]() {
        const int row = nb * 16 + (lane & 15) < p.V ? nb * 16 + (lane & 15) : p.V - 1;
        src = p.q + static_cast<long long>(row) * p.ldq + nk * (I4_CHUNK * 64);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int e = i * 32 + lane, r = nb * 16 + e / SC < p.V ? nb * 16 + e / SC : p.V - 1;
            sp[i] = static_cast<const T *>(p.scale) + static_cast<long long>(r) * p.lds + nk * SC + e % SC;
        }
    };
    rows_at();
    const uint32_t bar0 = smem_u32(&bars[warp][0]), to0 = smem_u32(mine) + (lane & 15) / 2 * I4_ROW + (lane & 1) * I4_ODD;
    auto bring = [&](int buf) {
        if (nc >= c_end) return;
        const int left = row_bytes - nk * (I4_CHUNK * 64);
        const int bytes = left < I4_CHUNK * 64 ? left : I4_CHUNK * 64;
        if (lane == 0) mbar_arrive_expect_tx(&bars[warp][buf], 16 * bytes);
        __syncwarp();
        if (lane < 16)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    to0 + buf * I4_BUF),
                "l"(src), "r"(bytes), "r"(bar0 + buf * 8)
                : "memory");
        src += I4_CHUNK * 64;
        const int ahead = groups - nk * SC;   // groups from this chunk on
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            sc[i] = 0.f;
            if ((i * 32 + lane) % SC < ahead && (16 * SC % 32 == 0 || i * 32 + lane < 16 * SC)) sc[i] = to_float(*sp[i]);
            sp[i] += SC;
        }
        ++nc;
        if (++nk == cpb) {
            nk = 0;
            ++nb;
            rows_at();
        }
    };
    auto keep_scales = [&](int buf) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (16 * SC % 32 == 0 || i * 32 + lane < 16 * SC) my_scales[buf * 16 * SC + i * 32 + lane] = sc[i];
    };
#pragma unroll
    for (int i = 0; i < I4_RING; ++i) {
        bring(i);
        if (i + 1 < I4_RING) keep_scales(i);
    }

    // x into shared memory, beside the first loads
    const T *X = static_cast<const T *>(p.X);
    if (std::is_same<T, __nv_bfloat16>::value) {
        const int per = (p.D + 255) / 256;   // steps of a warp over a token
#pragma unroll 4
        for (int i = warp; i < per * mt; i += warps) {
            const int m = i / per, k = i % per * 256 + lane * 8;
            const uint16_t *src = reinterpret_cast<const uint16_t *>(X) + static_cast<long long>(m) * p.ldx + k;
            uint32_t most = 0u;   // (finite bf16 magnitudes order as their bits do)
            if (p.x_vec && k + 8 <= p.D) {
                const uint4 q = *reinterpret_cast<const uint4 *>(src);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t v = (&q.x)[e / 2] >> (16 * (e & 1)) & 0x7fffu;
                    if (v < 0x7f80u && v > most) most = v;
                }
            } else {
                for (int e = 0; e < 8 && k + e < p.D; ++e) {
                    const uint32_t v = src[e] & 0x7fffu;
                    if (v < 0x7f80u && v > most) most = v;
                }
            }
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) atomicMax(&s_max[m], most);
        }
        __syncthreads();
        if (t < mt) {
            const float m = __uint_as_float(s_max[t] << 16);
            int e = 0;
            if (m > 0.f) frexpf(m, &e);   // m < 2^e
            const int up = m > 0.f ? (15 - e < 120 ? 15 - e : 120) : 0;
            s_up[t] = ldexpf(1.f, up);
            s_down[t] = ldexpf(1.f, -up);
        }
    } else if (t < 8) {
        s_up[t] = s_down[t] = 1.f;
    }
    __syncthreads();
    for (int i = t; i < units * 16 * mt; i += threads) {
        const int tt = i & 3, j = (i >> 2) & 3, m = (i >> 4) % mt, u = (i >> 4) / mt;
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
        if (std::is_same<T, __nv_bfloat16>::value) {
            const float up = s_up[m];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __half_as_ushort(__float2half_rn(__uint_as_float(static_cast<uint32_t>(v[e]) << 16) * up));
        }
        // pairs (0, 4), (1, 5), (2, 6), (3, 7): the order in which a word's nibbles come
        xw[(u * mt + m) * 16 + (j ^ (m & 1)) * 4 + tt] =
            make_uint4(v[0] | (v[4] << 16), v[1] | (v[5] << 16), v[2] | (v[6] << 16), v[3] | (v[7] << 16));
    }
    __syncthreads();

    float acc[4] = {}, head[4] = {};
    // a lane's pieces of x: where its even and its odd words are counted from (their order goes by the
    // token), and the step to the next unit's; lanes of no token read zeros
    const uint32_t x_at = smem_u32(g < mt ? xw + g * 16 + tl : zero);
    const uint32_t swap = g < mt ? (g & 1) * 64 : 0, xu = g < mt ? mt * 256 : 0;
    uint32_t magic;
    asm volatile("mov.u32 %0, 0x64006400;" : "=r"(magic));
    const uint32_t q_at = smem_u32(mine) + g / 2 * I4_ROW + (g & 1) * I4_ODD + tl * 16, s_at = smem_u32(my_scales) + g * (SC * 4);
    // a unit: its rows at qs, its scales at ss, its x at x0 (even words) and x1 (odd words)
    auto compute = [&](uint32_t qs, uint32_t ss, uint32_t x0, uint32_t x1) {
        const uint4 qa = lds128<0>(qs), qb = lds128<4 * I4_ROW>(qs);
        uint32_t q0[4] = {qa.x, qa.y, qa.z, qa.w}, q1[4] = {qb.x, qb.y, qb.z, qb.w};
        exchange<GROUP>(q0, tl);
        exchange<GROUP>(q1, tl);
        const uint4 x[4] = {lds128<0>(x0), lds128<64>(x1), lds128<128>(x0), lds128<192>(x1)};
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            float c[4], d[4];   // (two chains of products, half as long)
#pragma unroll
            for (int j = k * JS; j < (k + 1) * JS; ++j) {
                __half2 a[4], b[4];
                nibbles(q0[j], magic, a);
                nibbles(q1[j], magic, b);
                mma16816(c, a[0], b[0], a[1], b[1], x[j].x, x[j].y, j == k * JS);
                mma16816(d, a[2], b[2], a[3], b[3], x[j].z, x[j].w, j == k * JS);
            }
            const float s0 = lds32<0>(ss + k * 4), s1 = lds32<8 * SC * 4>(ss + k * 4);
            acc[0] = fmaf(s0, c[0] + d[0], acc[0]);
            acc[1] = fmaf(s0, c[1] + d[1], acc[1]);
            acc[2] = fmaf(s1, c[2] + d[2], acc[2]);
            acc[3] = fmaf(s1, c[3] + d[3], acc[3]);
        }
    };
    T *out = static_cast<T *>(p.out);
    bool ok = true;
    auto write = [&](int rb) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = 2 * tl + i;
            if (m < mt) {
                T *o = out + static_cast<long long>(m) * p.ldc + rb * 16ll + g;
                const float down = ok ? s_down[m] : NAN;   // (a wait for copies that ran out is not passed over)
                if (rb * 16 + g < p.V) o[0] = from_float<T>(acc[i] * down);
                if (rb * 16 + g + 8 < p.V) o[8] = from_float<T>(acc[i + 2] * down);
            }
        }
    };
    const int c_begin = begin_of(warp);
    int rb = b0 + c_begin / cpb, k = c_begin % cpb, buf = 0;
    bool from_start = k == 0;   // the row block at hand was begun at its first chunk
    uint32_t par = 0;
    for (int c = c_begin; c < c_end; ++c) {
        const uint32_t bar = smem_u32(&bars[warp][buf]);
        if (!mbar_try_wait(bar, par)) {
            const uint64_t t0 = global_timer_ns();
            while (ok && !mbar_try_wait(bar, par)) ok = global_timer_ns() - t0 <= I4_WAIT_NS;
            ok = __all_sync(0xffffffffu, ok);
        }
        __syncwarp();
        const int n = units - k * I4_CHUNK;
        uint32_t qs = q_at + buf * I4_BUF, ss = s_at + buf * (16 * SC * 4);
        uint32_t x0 = x_at + k * I4_CHUNK * xu + swap, x1 = x0 - 2 * swap;
        if (n >= I4_CHUNK) {
#pragma unroll
            for (int i = 0; i < I4_CHUNK; ++i) compute(qs + i * 64, ss + i * (PER * 4), x0 + i * xu, x1 + i * xu);
        } else {
#pragma unroll 1
            for (int i = 0; i < n; ++i) compute(qs + i * 64, ss + i * (PER * 4), x0 + i * xu, x1 + i * xu);
        }
        __syncwarp();
        keep_scales(buf == 0 ? I4_RING - 1 : buf - 1);      // (asked for a chunk ago)
        fence_proxy_async_smem();
        bring(buf);
        __syncwarp();
        if (++buf == I4_RING) {
            buf = 0;
            par ^= 1u;
        }
        if (++k == cpb) {
            if (from_start) write(rb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!from_start) head[i] = acc[i];
                acc[i] = 0.f;
            }
            k = 0;
            ++rb;
            from_start = true;
        }
    }
    // Row blocks that were shared: the warp that began one adds up the others' parts, in order: what
    // warps in the middle of it have (all theirs), then the end of it, which the last one began with.
    __syncthreads();
    float4 *part = reinterpret_cast<float4 *>(i4_smem);   // [warp][head, rest][lane], over the buffers
    part[(warp * 2 + 0) * 32 + lane] = make_float4(head[0], head[1], head[2], head[3]);
    part[(warp * 2 + 1) * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (c_begin < c_end && k > 0 && from_start) {
        const int end = (rb - b0 + 1) * cpb;   // the row block's last chunk and one
        for (int w = warp + 1; w < warps; ++w) {
            const bool whole = begin_of(w + 1) < end;
            if (begin_of(w) < begin_of(w + 1)) {
                const float4 o = part[(w * 2 + (whole ? 1 : 0)) * 32 + lane];
                acc[0] += o.x;
                acc[1] += o.y;
                acc[2] += o.z;
                acc[3] += o.w;
            }
            if (!whole) break;
        }
        write(rb);
    }
}

// ------------------------------------------------------------------ tokens on the 5th-generation tensor cores
// A CTA takes 128 rows of the weight (the A operand, in TMEM) times N tokens (B, in shared memory) over all of
// D, 256 values of k a stage:
//   * a producer warp brings the stage's packed rows (16 KB, 128-byte swizzle) and the tokens' values
//     (four boxes of 64 x N fp16) by TMA;
//   * two groups of four warps turn a half of the stage each into fp16 q - 8: a thread has a row, whose 64
//     bytes become 64 TMEM columns (as above; the k order within eight is that of a word's nibble pairs,
//     and the tokens were laid out in that order before);
//   * one warp issues the products: those of a group of k into a TMEM buffer of its own;
//   * eight warps read the groups' sums (a thread has a row and half of the tokens), scale them by the
//     row's scale of that group and add them up in fp32 registers.
// TMEM: columns 0-255 the sums' buffers, in two sets that are handed over as a whole, 256-511 two stages of A.
// A product of 128 x N x 16 takes some 50 cycles up to N = 96, so for few tokens a stage's sixteen take a little
// longer than its bytes (measured rates: 850 and 700 cycles). What the issuing warp does per stage
// counts: with 128 values a stage and every barrier of its own, 16 tokens of 4096 x 128256 took 172 us.

constexpr int I4T_THREADS = 18 * 32;    // 8 warps of sums, 8 of values, the producer, the MMA warp
constexpr int I4T_Q = 16384;            // bytes of a stage's packed rows
constexpr int I4T_MAX_STAGES = 9;
constexpr int I4T_PRODUCER = 16, I4T_MMA = 17;

__device__ __forceinline__ void umma_f16_ta(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate));
}
// 32 columns of the warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// NH: tokens of a thread (half of the tile's N); PER: groups of 128 values.
template <int NH, int PER>
__global__ void __launch_bounds__(I4T_THREADS, 1) lce_int4_kernel(const __grid_constant__ Int4TileParams p) {
    constexpr int N = 2 * NH;
    constexpr int DCOLS = N <= 32 ? 32 : N <= 64 ? 64 : 128;
    constexpr int GROUPS = 2 * PER;                              // of a stage
    constexpr int STEPS = 16 / GROUPS;                           // products of a group
    constexpr int SET = GROUPS < 128 / DCOLS ? GROUPS : 128 / DCOLS;   // buffers that are handed over together
    constexpr int SETS = GROUPS / SET;                           // of a stage
    constexpr int STAGE = I4T_Q + N * 512;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[I4T_MAX_STAGES];    // a stage's bytes landed
    __shared__ __align__(8) uint64_t done_bar[I4T_MAX_STAGES];    // its products have ended: its bytes and its A are free
    __shared__ __align__(8) uint64_t afull_bar[2];                // its values are in TMEM
    __shared__ __align__(8) uint64_t dfull_bar[2];                // a set's sums are there
    __shared__ __align__(8) uint64_t dempty_bar[2];
    __shared__ __align__(8) uint64_t drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ int s_issued;   // stages that were asked for

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nstages = p.stages;
    if (threadIdx.x == 0) {
        for (int i = 0; i < nstages; ++i) {
            mbar_init(&full_bar[i], 1);
            mbar_init(&done_bar[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull_bar[i], 8);
            mbar_init(&dfull_bar[i], 1);
            mbar_init(&dempty_bar[i], 8);
        }
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == I4T_PRODUCER && lane == 0) {
        prefetch_tmap(&p.tmQ);
        prefetch_tmap(&p.tmX);
    }
    if (warp == I4T_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    Abort ab;
    ab.flag_smem = &abort_flag;
    ab.hdr = p.hdr;
    ab.limit_ns = p.timeout_ns;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // (the tokens' layout has been written)

    const int items = p.row_tiles * p.token_tiles, nk = (p.units + 1) / 2;
    const int mine = static_cast<int>(blockIdx.x) < items ? (items - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1 : 0;
    const int total = mine * nk;   // stages of this CTA
    if (warp == I4T_PRODUCER) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int t = p.bring ? static_cast<int>(blockIdx.x) : items; ok && t < items; t += gridDim.x) {
                const int row0 = t / p.token_tiles * 128, m0 = t % p.token_tiles * N;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(&done_bar[stage], phase, ab)) {
                        ok = false;
                        break;
                    }
                    uint8_t *to = smem + stage * STAGE;
                    mbar_arrive_expect_tx(&full_bar[stage], STAGE);
                    tma_load_2d(to, &p.tmQ, &full_bar[stage], kb * 128, row0);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        tma_load_2d(to + I4T_Q + b * (N * 128), &p.tmX, &full_bar[stage], kb * 256 + b * 64, m0);
                    ++issued;
                    if (++stage == nstages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            s_issued = issued;
        }
    } else if (warp == I4T_MMA) {
        // (the whole warp goes along; one lane issues)
        int stage = 0;
        uint32_t phase = 0, aphase = 0, dphase = 1;   // (a set's phase: sets alternate, so both flip every second one)
        bool ok = true, any = false;
        // D fp32, A and B fp16, both K-major
        constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
        int half = 0, set = 0;
        for (int it = 0; it < total; ++it) {
            const uint64_t bd = sdesc(smem_u32(smem + stage * STAGE + I4T_Q), 16u, 1024u);
            const uint32_t a = tmem + 256 + half * 128;
            ok = mbar_wait(&full_bar[stage], phase, ab) && mbar_wait(&afull_bar[half], aphase, ab);
#pragma unroll
            for (int c = 0; c < SETS; ++c) {
                const uint32_t d = tmem + set * 128;
                ok = __all_sync(0xffffffffu, ok && mbar_wait(&dempty_bar[set], dphase, ab));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int g = 0; g < SET; ++g)
#pragma unroll
                        for (int j = 0; j < STEPS; ++j) {
                            const int k = (c * SET + g) * STEPS + j;   // of the stage's sixteen
                            umma_f16_ta(d + g * DCOLS, a + k * 8,
                                        bd + static_cast<uint64_t>(k / 4 * (N * 128 / 16) + k % 4 * 2), idesc,
                                        j ? 1u : 0u);
                        }
                    umma_commit(&dfull_bar[set]);
                    if (c + 1 == SETS) umma_commit(&done_bar[stage]);
                }
                __syncwarp();
                any = true;
                set ^= 1;
                if (set == 0) dphase ^= 1;
            }
            if (!ok) break;
            if (++stage == nstages) {
                stage = 0;
                phase ^= 1;
            }
            half ^= 1;
            if (half == 0) aphase ^= 1;
        }
        if (any) {   // every product has ended before TMEM is given back
            if (elect_one()) umma_commit(&drain_bar);
            __syncwarp();
            mbar_wait_drain(&drain_bar, 0, 50000000ull);
        }
    } else if (warp >= 8) {
        // values: this group's half of every stage
        const int unit = (warp - 8) >> 2, row = (warp & 3) * 32 + lane;
        uint32_t magic;
        asm volatile("mov.u32 %0, 0x64006400;" : "=r"(magic));
        const uint32_t to0 = tmem + 256 + unit * 64 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        int stage = 0, old = nstages - 2, half = 0;   // old: the stage that had this half of A before
        uint32_t phase = 0, ophase = 1;
        for (int it = 0; it < total; ++it) {
            bool ok = mbar_wait(&full_bar[stage], phase, ab) && (it < 2 || mbar_wait(&done_bar[old], ophase, ab));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t at = smem_u32(smem + stage * STAGE) + row * 128;
            const uint32_t turn = (row & 7) << 4;
            uint4 q[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) q[c] = lds128<0>(at + (((unit * 4 + c) << 4) ^ turn));
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    __half2 v[4];
                    nibbles((&q[2 * h + j / 4].x)[j % 4], magic, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[4 * j + i] = *reinterpret_cast<uint32_t *>(&v[i]);
                }
                tmem_st32(to0 + half * 128 + h * 32, r);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&afull_bar[half]);
            if (++stage == nstages) {
                stage = 0;
                phase ^= 1;
            }
            if (++old == nstages) {
                old = 0;
                ophase ^= 1;
            }
            half ^= 1;
        }
    } else {
        // sums
        const int half = warp >> 2, row_in = (warp & 3) * 32 + lane;
        const uint32_t at0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * NH;
        int set = 0;
        uint32_t dphase = 0;
        bool ok = true;
        const int groups = p.groups;
        for (int t = blockIdx.x; ok && t < items; t += gridDim.x) {
            const int row = t / p.token_tiles * 128 + row_in, m0 = t % p.token_tiles * N + half * NH;
            const uint16_t *sp = static_cast<const uint16_t *>(p.scale) +
                                 static_cast<long long>(row < p.V ? row : p.V - 1) * p.lds;
            float2 acc[NH / 2];
#pragma unroll
            for (int j = 0; j < NH / 2; ++j) acc[j] = make_float2(0.f, 0.f);
            // a set's scales are asked for two sets ahead
            uint16_t ahead[2][SET];
            auto ask = [&](uint16_t (&o)[SET], int g) {
#pragma unroll
                for (int i = 0; i < SET; ++i) o[i] = g + i < groups ? sp[g + i] : static_cast<uint16_t>(0);
            };
            ask(ahead[0], 0);
            ask(ahead[1], SET);
            const int all = nk * GROUPS;
            for (int g0 = 0; ok && g0 < all; g0 += 2 * SET) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (!ok || g0 + c * SET >= all) continue;
                    float s[SET];
#pragma unroll
                    for (int i = 0; i < SET; ++i)
                        s[i] = p.dtype == CE_FP16 ? __half2float(__ushort_as_half(ahead[c][i]))
                                                  : __uint_as_float(static_cast<uint32_t>(ahead[c][i]) << 16);
                    ask(ahead[c], g0 + (2 + c) * SET);
                    ok = __all_sync(0xffffffffu, mbar_wait(&dfull_bar[set], dphase, ab));
                    if (!ok) continue;
                    tc_fence_after();
// pieces of eight columns, four under way at a time
                    constexpr int PIECES = SET * NH / 8;
#pragma unroll
                    for (int b = 0; b < PIECES; b += 4) {
                        uint32_t v[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (b + j < PIECES)
                                tmem_ld8(at0 + set * 128 + (b + j) / (NH / 8) * DCOLS + (b + j) % (NH / 8) * 8, v + 8 * j);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(v[j]));
                        if (b + 4 >= PIECES) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&dempty_bar[set]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (b + j < PIECES) {
                                const float si = s[(b + j) / (NH / 8)];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float2 &o = acc[(b + j) % (NH / 8) * 4 + e];
                                    o = __ffma2_rn(make_float2(__uint_as_float(v[8 * j + 2 * e]),
                                                               __uint_as_float(v[8 * j + 2 * e + 1])),
                                                   make_float2(si, si), o);
                                }
                            }
                    }
                    set ^= 1;
                    if (set == 0) dphase ^= 1;
                }
            }
            if (row < p.V && ok) {
                uint16_t *out = static_cast<uint16_t *>(p.out) + row;
#pragma unroll
                for (int j = 0; j < NH; ++j)
                    if (m0 + j < p.M) {
                        const float v = (j & 1 ? acc[j / 2].y : acc[j / 2].x) * p.down[m0 + j];
                        out[static_cast<long long>(m0 + j) * p.ldc] =
                            p.dtype == CE_FP16 ? __half_as_ushort(__float2half_rn(v))
                                               : __bfloat16_as_ushort(__float2bfloat16_rn(v));
                    }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // After a wait that ran out, whosever it was: the copies still in flight end (bounded) before the shared memory is given
    // back; and NaN in all tiles of this CTA, since nobody may ask for the status. (Here, where nothing is kept any
    // more: among the sums' results, 192 tokens x 128256 x 4096 took 268 us in place of 237.)
    if (abort_flag) {
        if (threadIdx.x == 0)
            for (int j = s_issued > nstages ? s_issued - nstages : 0; j < s_issued; ++j)
                mbar_wait_drain(&full_bar[j % nstages], static_cast<uint32_t>((j / nstages) & 1), 50000000ull);
#pragma unroll 1
        for (int t = blockIdx.x; t < items; t += gridDim.x) {
            const int row0 = t / p.token_tiles * 128, m0 = t % p.token_tiles * N;
#pragma unroll 1
            for (int i = threadIdx.x; i < 128 * N; i += I4T_THREADS)
                if (row0 + i % 128 < p.V && m0 + i / 128 < p.M)
                    static_cast<uint16_t *>(p.out)[static_cast<long long>(m0 + i / 128) * p.ldc + row0 + i % 128] =
                        0x7fff;   // (a NaN in both types)
        }
    }
    if (warp == I4T_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// The tokens for it: a CTA per token; fp16 (bf16 brought below 2^15 by a power of two), eight values in the order 0 4 1
// 5 2 6 3 7, rows filled up with zeros to whole units.
constexpr int I4X_THREADS = 256;

template <typename T>
__global__ void __launch_bounds__(I4X_THREADS) lce_int4_tokens_kernel(const Int4TileParams p, const T *X, long long ldx,
                                                                      int x_vec, uint4 *to) {
    __shared__ unsigned s_max;
    const int t = threadIdx.x, m = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;");
    if (m == 0 && t < HDR_COUNTERS) p.hdr[t] = 0;
    const uint16_t *src = reinterpret_cast<const uint16_t *>(X + m * ldx);
    auto load = [&](int k, uint16_t (&v)[8]) {
        if (x_vec && k + 8 <= p.D) {
            const uint4 q = *reinterpret_cast<const uint4 *>(src + k);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = static_cast<uint16_t>((&q.x)[e / 2] >> (16 * (e & 1)));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = k + e < p.D ? src[k + e] : static_cast<uint16_t>(0);
        }
    };
    float up = 1.f, down = 1.f;
    if (std::is_same<T, __nv_bfloat16>::value) {
        if (t == 0) s_max = 0u;
        __syncthreads();
        uint32_t most = 0u;   // (finite bf16 magnitudes order as their bits do)
        for (int k = t * 8; k < p.D; k += I4X_THREADS * 8) {
            uint16_t v[8];
            load(k, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t a = v[e] & 0x7fffu;
                if (a < 0x7f80u && a > most) most = a;
            }
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if ((t & 31) == 0) atomicMax(&s_max, most);
        __syncthreads();
        const float a = __uint_as_float(s_max << 16);
        int e = 0;
        if (a > 0.f) {
            frexpf(a, &e);   // a < 2^e
            e = 15 - e < 120 ? 15 - e : 120;
        }
        up = ldexpf(1.f, e);
        down = ldexpf(1.f, -e);
    }
    if (t == 0) p.down[m] = down;
    for (int i = t; i < p.units * 16; i += I4X_THREADS) {
        uint16_t v[8];
        load(i * 8, v);
        if (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __half_as_ushort(__float2half_rn(__uint_as_float(static_cast<uint32_t>(v[e]) << 16) * up));
        }
        to[static_cast<long long>(m) * p.units * 16 + i] =
            make_uint4(v[0] | (v[4] << 16), v[1] | (v[5] << 16), v[2] | (v[6] << 16), v[3] | (v[7] << 16));
    }
}

// ------------------------------------------------------------------ quantisation
// A warp per row and 256 values: a lane's eight values, the maximum over the lanes of a group.

constexpr int I4Q_THREADS = 256;

template <typename S> struct ScaleRange;
template <> struct ScaleRange<__nv_bfloat16> {
    static constexpr float smallest = 0x1p-133f, largest = 0x1.fep127f;
};
template <> struct ScaleRange<__half> {
    static constexpr float smallest = 0x1p-24f, largest = 65504.f;
};

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
    // a seventh of the largest magnitude, as the scale's type has it, within its smallest and largest positive
    // number (fp16 has neither a seventh of 1e-7 nor of 1e6): values beyond are -8 or 7 of the largest, and
    // those below half the smallest are 0; a group that holds an infinity or a NaN gets a NaN
    using Range = ScaleRange<S>;
    const S s16 = from_float<S>(fminf(fmaxf(amax / 7.f, Range::smallest), Range::largest));
    const float s = amax > 0.f ? to_float(s16) : 1.f;
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

template <typename T>
cudaError_t launch_few_of(const Int4Params &p, dim3 grid, int threads, size_t smem, cudaStream_t s) {
    if (p.group == 128) lce_int4_few_kernel<T, 128><<<grid, threads, smem, s>>>(p);
    else if (p.group == 64) lce_int4_few_kernel<T, 64><<<grid, threads, smem, s>>>(p);
    else lce_int4_few_kernel<T, 32><<<grid, threads, smem, s>>>(p);
    return cudaGetLastError();
}

constexpr int I4_MAX_SMEM = 220 * 1024;

// Shared memory of x for so many tokens, and of a warp.
size_t few_x_smem(const Int4Params &p, int tokens) { return 256 + static_cast<size_t>(p.units) * 256 * tokens; }
size_t few_warp_smem(const Int4Params &p) { return I4_RING * (I4_BUF + 16 * 4 * I4_CHUNK * (I4_UNIT / p.group)); }

template <typename T, int GROUP> cudaError_t set_few() {
    return cudaFuncSetAttribute(lce_int4_few_kernel<T, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, I4_MAX_SMEM);
}

template <int NH, int PER> cudaError_t set_tile() {
    return cudaFuncSetAttribute(lce_int4_kernel<NH, PER>, cudaFuncAttributeMaxDynamicSharedMemorySize, I4_MAX_SMEM);
}
template <int NH> cudaError_t set_tiles() {
    cudaError_t e;
    if ((e = set_tile<NH, 1>()) != cudaSuccess) return e;
    if ((e = set_tile<NH, 2>()) != cudaSuccess) return e;
    return set_tile<NH, 4>();
}
template <int NH> cudaError_t launch_tiles_of(const cudaLaunchConfig_t &cfg, const Int4TileParams &p) {
    return p.per == 1   ? cudaLaunchKernelEx(&cfg, lce_int4_kernel<NH, 1>, p)
           : p.per == 2 ? cudaLaunchKernelEx(&cfg, lce_int4_kernel<NH, 2>, p)
                        : cudaLaunchKernelEx(&cfg, lce_int4_kernel<NH, 4>, p);
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
    if ((e = set_few<__half, 32>()) != cudaSuccess) return e;
    if ((e = set_tiles<8>()) != cudaSuccess) return e;
    if ((e = set_tiles<16>()) != cudaSuccess) return e;
    if ((e = set_tiles<24>()) != cudaSuccess) return e;
    if ((e = set_tiles<32>()) != cudaSuccess) return e;
    return set_tiles<48>();
}

// Whether so many tokens go by the kernel for few. Measured at 128256 x 4096, bf16 (us; tiles / few): groups of
// 128: 1 token 70 / 62, 2: 71 / 66, 4: 71 / 75; of 64: 1: 90 / 76, 4: 91 / 84; of 32: 1: 153 / 95, 6: 153 / 102, 8 (two
// passes): 154 / 193. The rule goes by tokens and groups alone: other D and V were not measured on both sides. Rows so
// long that the tokens do not fit beside eight warps' buffers go by tiles too.
bool int4_few(long long M, long long D, int group) {
    if (M > (group == 128 ? 2 : group == 64 ? 4 : 6)) return false;
    Int4Params p;
    p.units = static_cast<int>((D + I4_UNIT - 1) / I4_UNIT);
    p.group = group;
    return M == 1 || few_x_smem(p, static_cast<int>(M)) + 8 * few_warp_smem(p) <= I4_MAX_SMEM;
}

cudaError_t launch_int4(Int4Params p, int sms, cudaStream_t s) {
    p.units = (p.D + I4_UNIT - 1) / I4_UNIT;
    // as many warps as there is room for
    const size_t ws = few_warp_smem(p);
    const long long room = (static_cast<long long>(I4_MAX_SMEM) - static_cast<long long>(few_x_smem(p, p.M))) /
                           static_cast<long long>(ws);
    if (room < 1) return cudaErrorInvalidValue;
    const int warps = room < I4_MAX_WARPS ? static_cast<int>(room) : I4_MAX_WARPS;
    const int blocks = (p.V + 15) / 16;
    const dim3 grid(blocks < sms ? blocks : sms);
    const size_t smem = few_x_smem(p, p.M) + warps * ws;
    return p.dtype == CE_FP16 ? launch_few_of<__half>(p, grid, warps * 32, smem, s)
                              : launch_few_of<__nv_bfloat16>(p, grid, warps * 32, smem, s);
}

// Tokens of a tile for M of them, and tiles.
int int4_tile_tokens(long long M) {
    const long long tiles = (M + 95) / 96, n = (M + tiles - 1) / tiles;
    return n <= 16 ? 16 : n <= 32 ? 32 : n <= 48 ? 48 : n <= 64 ? 64 : 96;
}

cudaError_t launch_int4_tokens(const Int4TileParams &p, const void *X, long long ldx, int x_vec, void *to, cudaStream_t s) {
    if (p.dtype == CE_FP16)
        lce_int4_tokens_kernel<__half><<<p.M, I4X_THREADS, 0, s>>>(p, static_cast<const __half *>(X), ldx, x_vec, static_cast<uint4 *>(to));
    else
        lce_int4_tokens_kernel<__nv_bfloat16><<<p.M, I4X_THREADS, 0, s>>>(p, static_cast<const __nv_bfloat16 *>(X), ldx, x_vec,
                                                                         static_cast<uint4 *>(to));
    return cudaGetLastError();
}

cudaError_t launch_int4_tiles(Int4TileParams p, int n, int sms, cudaStream_t s) {
    const int stage = I4T_Q + n * 512;
    p.stages = (I4_MAX_SMEM - 1024) / stage < I4T_MAX_STAGES ? (I4_MAX_SMEM - 1024) / stage : I4T_MAX_STAGES;
    const int items = p.row_tiles * p.token_tiles;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(items < sms ? items : sms);
    cfg.blockDim = dim3(I4T_THREADS);
    cfg.dynamicSmemBytes = I4_MAX_SMEM;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    switch (n) {
        case 16: return launch_tiles_of<8>(cfg, p);
        case 32: return launch_tiles_of<16>(cfg, p);
        case 48: return launch_tiles_of<24>(cfg, p);
        case 64: return launch_tiles_of<32>(cfg, p);
        default: return launch_tiles_of<48>(cfg, p);
    }
}

cudaError_t launch_int4_quantize(const Int4QuantParams &p, cudaStream_t s) {
    return p.dtype == CE_FP32 ? launch_quant<float>(p, s)
           : p.dtype == CE_FP16 ? launch_quant<__half>(p, s) : launch_quant<__nv_bfloat16>(p, s);
}

}  // namespace lce
