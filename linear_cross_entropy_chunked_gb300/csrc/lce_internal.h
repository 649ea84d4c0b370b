// Internal declarations shared by the kernels and the C-ABI host code.
// Not part of the public interface (that is include/lce.h).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lce {

// ---------------------------------------------------------------- GEMM tiling
// One CTA per SM, persistent. A 128 x 256 fp32 accumulator tile lives in TMEM
// (256 columns); two of them (512 columns = all of TMEM) let the epilogue of
// tile t overlap the MMAs of tile t+1.
constexpr int BM = 128;            // UMMA M (TMEM lanes)
constexpr int BN = 256;            // UMMA N (TMEM columns per accumulator)
constexpr int BK = 64;             // one 128-byte swizzle row of bf16
constexpr int UMMA_K = 16;         // K of one tcgen05.mma kind::f16
constexpr int A_BYTES = BM * BK * 2;             // 16 KB
constexpr int B_BYTES = BN * BK * 2;             // 32 KB
// Pipeline per CTA. One CTA per tile: 4 stages of A (16 KB) + B (32 KB). CTA
// pair on one 256 x 256 tile (tcgen05 cta_group::2): each CTA holds its own A
// rows and half of B, 6 stages of 16 + 16 KB.
// Pipeline stages: A (128 rows x 64) plus this CTA's share of B. WIDE: the
// CTA-pair dH tiles 512 columns wide (two N = 256 MMAs share A), whose stage
// carries two B halves.
template <int CL, bool WIDE = false> struct Pipe {
    static constexpr int kBBytes = (WIDE ? 2 : 1) * B_BYTES / CL;
    static constexpr int kStageBytes = A_BYTES + kBBytes;
    static constexpr int kStages = (4 * 48 * 1024) / kStageBytes;
};
constexpr int MAX_STAGES = 6;
constexpr int STAGES = 4;                                  // one-CTA pipeline
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;             // 48 KB
constexpr int STAGING_BYTES = 16384;  // per epilogue column half: one 128-row x 128-byte store box
constexpr int PIPE_BYTES = 4 * 48 * 1024;      // both pipelines use 192 KB
constexpr int GEMM_SMEM_BYTES = PIPE_BYTES + 2 * STAGING_BYTES + 1024;  // + 1 KB alignment
constexpr int NUM_EPI_WARPS = 8;   // warps 0..7: TMEM lane quarter = warp % 4, column half = warp / 4
constexpr int PRODUCER_WARP = 8;
constexpr int MMA_WARP = 9;
constexpr int GEMM_THREADS = 320;
constexpr int SCHED_DEPTH = 4;
constexpr int TMEM_COLS = 512;
constexpr int BN_WIDE = 512;   // MODE_DH tile width: both 256-column TMEM accumulators
// dH tiles (256 rows x 512 columns on a CTA pair) run over the whole vocabulary
// while the dW tiles, whose 256 x 256 shape needs more operand bytes per flop
// and which also stage and reduce-add their fp32 output, run concurrently on the
// other SMs. The phase is shortest when both sets end together: measured on a
// GB300 that is about 32 dH tiles (a dH tile pair runs ~1.3x the flop rate of a
// dW one; 76 pairs). A chunk with fewer dH tiles splits them along the
// vocabulary until there are at least DH_SPLIT_TILES, in at most DH_MAX_SPLITS
// parts, for vocabularies of at least DH_SPLIT_MIN_V; more dH tiles than that
// leave the dW tiles to the end of the phase (measured slower, both with one dW
// contraction per chunk and per pair of chunks).
constexpr int DH_SPLIT_TILES = 28;
constexpr int DH_MAX_SPLITS = 4;
constexpr long long DH_SPLIT_MIN_V = 8192;
constexpr int PART_COLS = 128;     // columns covered by one (max, sum) partial

// Epilogue / tile-set modes of the GEMM kernel.
enum GemmMode : int {
    MODE_LSE = 0,     // logits tiles -> per-(row, 128-col) (max, sumexp) partials + target logit
    MODE_LSE_P = 1,   // ... + store P' = exp(z - max_part) as bf16 into the chunk buffer
    MODE_G = 2,       // logits tiles -> G = (exp(z - lse) - onehot) * scale as bf16 (given lse)
    MODE_BWD = 3,     // dH tiles (G W) followed by dW tiles (G^T H) in one persistent launch
    MODE_DH = 4       // dH tiles only, 256 rows x 512 columns per CTA pair (CTA pairs only)
};

// Scale of row i of G: dloss (a scalar, or row i of a per-row vector) divided
// by N_valid for the mean reduction; 0 for rows that do not count.
__device__ __forceinline__ float lce_row_scale(const float *dloss, int dloss_per_row, int mean,
                                               int n_valid, long long grow, bool y_ok) {
    if (!y_ok) return 0.f;
    const float d = dloss ? dloss[dloss_per_row ? grow : 0] : 1.f;
    if (mean) return n_valid > 0 ? d / static_cast<float>(n_valid) : 0.f;
    return d;
}

// fp16 inputs: G is stored in fp16, where dloss / N_valid (~1e-4 at the
// workloads' sizes) would push it below the format's range. So for fp16 the
// stored G is (p - onehot) * F16_G_SCALE (|G| <= 2^14), and the gradient
// epilogues multiply the dH / dW accumulators by (dloss / N_valid) / F16_G_SCALE
// (reduction mean; dloss / F16_G_SCALE for sum). bf16 keeps the full scale in G.
constexpr float F16_G_SCALE = 16384.f;

// Scale of row i of the stored G.
__device__ __forceinline__ float lce_store_scale(const float *dloss, int dloss_per_row, int mean,
                                                 int n_valid, long long grow, bool y_ok, int f16) {
    if (!f16) return lce_row_scale(dloss, dloss_per_row, mean, n_valid, grow, y_ok);
    return y_ok ? F16_G_SCALE : 0.f;
}

// Factor the gradient epilogues apply to their accumulators (1 for bf16).
__device__ __forceinline__ float lce_out_scale(const float *dloss, int mean, int n_valid, int f16) {
    if (!f16) return 1.f;
    const float d = dloss ? dloss[0] : 1.f;
    if (mean) return n_valid > 0 ? d / (static_cast<float>(n_valid) * F16_G_SCALE) : 0.f;
    return d / F16_G_SCALE;
}

// The clipped policy loss (lce_policy_*): what the log probability of a row's label is
// worth, in place of the cross-entropy. Null pointers: no such term.
struct PolicyParams {
    const float *adv;          // [N] advantages; null: the row loss is the cross-entropy
    const float *old_logp;     // [N] or null (the ratio is 1)
    const float *ref_logp;     // [N] or null (no KL term)
    const float *weight;       // [N] or null (1)
    float lo, hi;              // the ratio is held between them: 1 - clip_low, 1 + clip_high
    float beta;                // of the KL term (0: ref_logp is not read)
    float inv_t;               // 1 / temperature of the softmax
    float *logp;               // [N] output: log probability of the label, 0 where the row does not count
};

// Loss of a counting row and its derivative by the label's log probability, both times the
// row's weight:
//   r = exp(logp - old), f = r A, h = clamp(r, lo, hi) A
//   loss  = -min(f, h) + beta (e^d - 1 - d),  d = ref - logp
//   slope = -(f <= h ? f : 0) - beta (e^d - 1)
// The ratio is compared, not passed through min and max, so that a NaN stays one; an advantage
// of 0 gives 0 even where the ratio overflows.
struct PolicyRow {
    float loss, slope;
};
struct PolicyInputs {   // of a row
    float a, old_logp, ref_logp, w;
};
__device__ __forceinline__ PolicyInputs lce_policy_inputs(const PolicyParams &p, long long i) {
    return PolicyInputs{p.adv ? p.adv[i] : 0.f, p.old_logp ? p.old_logp[i] : 0.f,
                        p.ref_logp ? p.ref_logp[i] : 0.f, p.weight ? p.weight[i] : 1.f};
}
__device__ __forceinline__ PolicyRow lce_policy_row(const PolicyParams &p, const PolicyInputs &x, float logp) {
    const float r = p.old_logp ? expf(logp - x.old_logp) : (logp == logp ? 1.f : logp);
    const float f = r * x.a;
    const float h = (r < p.lo ? p.lo : r > p.hi ? p.hi : r) * x.a;
    PolicyRow o;
    o.loss = f <= h ? -f : -h;
    o.slope = f <= h ? -f : h * 0.f;
    if (p.ref_logp && p.beta != 0.f) {
        const float d = x.ref_logp - logp;
        const float e = expm1f(d);
        o.loss += p.beta * (d == INFINITY ? d : e - d);
        o.slope -= p.beta * e;
    }
    o.loss *= x.w;
    o.slope *= x.w;
    return o;
}
__device__ __forceinline__ PolicyRow lce_policy_row(const PolicyParams &p, long long i, float logp) {
    return lce_policy_row(p, lce_policy_inputs(p, i), logp);
}

// Losses on answers keep what the rounding of G to bf16 leaves of each row's label entry, (p - 1) scale: where the label is
// unlikely that entry is nearly all of the row, and half a step of it (2^-9) would be missing from dH's
// whole row and from dW's row of the label. The remainders are added in fp32: rest W[y] to the row of
// dH (in the gradient's epilogue, or where the rows are taken to their places), and, in the epilogue, to dW's row v those of the rows whose label it is, from first[v] on by next, REST_ROWS of them at
// most (of more rows the roundings average out, and one thread would have them all to do).
constexpr int REST_ROWS = 8;
struct LabelRests {
    float *rest;           // [rows of a chunk]; null: not kept
    int *first;            // [V]: the first row of the chunk with that label, or -1
    int *next;             // [rows of a chunk]
};
__device__ __forceinline__ float lce_rest(float g) {
    const float e = g - __bfloat162float(__float2bfloat16_rn(g));
    return fabsf(e) < INFINITY ? e : 0.f;
}

// Losses on answers at a temperature T: P' and the sum of a slab of 128 logits are relative to the slab's largest
// logit m, as powers of two to z k2 - m k2, k2 = log2(e) / T, with m k2 as fp32 rounds it: one fused operation a
// logit. That rounding is half a unit of m k2, up to an eighth below 2^22; from there on (T = 1e-6) the distance z - m is formed first.
// The slab's maximum is kept as it is, and whoever merges slabs subtracts what their base was short of m k2:
constexpr float BASE_ROUNDED_BELOW = 0x1p22f;
__device__ __forceinline__ float lce_base_rest(float m, float k2) {
    const float base = m * k2;
    return fabsf(base) < BASE_ROUNDED_BELOW ? fmaf(m, k2, -base) : 0.f;
}

// Workspace header (int32 words).
enum : int {
    HDR_FLAG = 0,       // bit 0: label out of range, bit 1: pipeline wait timed out
    HDR_NVALID = 1,
    HDR_DONE = 2,       // parts of a launch that have finished (the last one adds up the loss)
    HDR_COUNTERS = 16,  // one dynamic tile counter per GEMM launch of a call
};
constexpr int FLAG_LABEL = 1;
constexpr int FLAG_TIMEOUT = 2;
constexpr int FLAG_OFFSETS = 4;   // offsets of sequences that decrease or leave the rows

struct GemmParams {
    CUtensorMap tmA0;      // logits A = H (K-major) | dH A = G (K-major)
    CUtensorMap tmB0;      // logits B = W (K-major) | dH B = W (MN-major)
    CUtensorMap tmA1;      // dW A = G^T, read from the chunk buffer G [C][ldg] (MN-major;
                           // 3-D: {64 columns, rows, 64-column blocks})
    CUtensorMap tmB1;      // dW B = H chunk^T [D][C] (K-major)
    CUtensorMap tmS0;      // output store: P' / G chunk buffer (bf16) | dH chunk (bf16)
    CUtensorMap tmS1;      // dW output store / reduce-add (fp32)
    int m_blocks0, n_blocks0, k_blocks0;
    int m_blocks1, n_blocks1, k_blocks1;   // dW tiles (0 in logits launches)
    int total_tiles;       // scheduling units: tiles, or tile pairs for CTA pairs
    int rows;              // rows in this chunk
    int row0;              // first global row of this chunk
    int a_row0;            // logits: row coordinate of the chunk's first row in the H map
    int V, D;
    long long ignore_index;
    const long long *y;    // labels, global [N]
    int *tile_counter;
    int *hdr;
    const float *dloss;    // device scalar, per-row vector, or null (= 1)
    int dloss_per_row;     // 1: dloss[N] (reduction none)
    int mean;              // 1: G scaled by 1 / N_valid (reduction mean)
    // logits epilogue
    float2 *parts;         // [rows][nparts] (max, sumexp)
    int nparts;
    float *zy;             // [rows] target logits
    __nv_bfloat16 *G;      // [rows][ldg] P' or G
    int ldg;
    const float *lse;      // global [N] (MODE_G)
    // backward epilogues
    __nv_bfloat16 *dH;     // global [N][D]
    float *dW;             // [V][D]
    int dw_accumulate;     // 0: store, 1: add to existing dW
    int dh_fp32;           // 1: dH tiles stored as fp32 (tmS0 an fp32 map)
    int dw_16;             // 1: dW stored as bf16 (tmS1 a bf16 map; not added to)
    LabelRests rests;      // (written by the G epilogue, read by the gradients' epilogues)
    const uint4 *Hc, *W;   // with rests: the chunk's rows of H, and W
    // dH launches: the vocabulary (K) range of every dH tile split in k_splits
    // parts of kb_per_split k blocks; part s stores fp32 partial sums at row
    // offset s * split_rows of the tmS0 map (k_splits <= 1: one part, no offset)
    int k_splits, kb_per_split, split_rows;
    int f16;               // 1: fp16 operands (H, W, G) and fp16 P' / G / dH stores
    int answers;           // 1: a loss on answers; what follows up to the wait's limit is read then only
    float inv_t;           // 1 / temperature: the logits epilogues form exp((z - m) inv_t)
    // Rows that count brought together (null: all `rows` are there): their number on the device. Tiles and
    // contractions then end with the rows there are; dw_row0 and dw_rows: the rows of the dW contraction.
    const int *counting;
    int dw_row0, dw_rows;
    unsigned long long timeout_ns;
};

struct MergeParams {
    const float2 *parts;   // [rows][nparts] (max, sumexp) per 128-column slab
    int nparts;
    float inv_t;           // losses on answers: 1 / temperature (maxima and zy are logits, sums those of exp((z - m) / T))
    const float *zy;
    const float *zx;       // null, or [rows]: the label's logit as an fp32 dot product of its own (zy: the tensor cores'),
    float2 *fix;           // for which [N] gets what the row's log probability moves by with it: (1 - p) (zx - zy, 1)
    __nv_bfloat16 *G;
    int ldg;
    int rows, row0, V;
    long long ignore_index;
    const long long *y;
    const int *hdr;
    const float *dloss;
    int dloss_per_row;
    int mean;
    int f16;               // fp16 inputs: slab factors use lce_store_scale
    float *lse;            // global [N]; null: not written
    float *loss_rows;      // global [N] (the caller's loss vector for reduction none)
    PolicyParams pol;      // pol.adv: the policy loss in place of the cross-entropy
    int answers;           // 1: a loss on answers
    // rows that count brought together: their number (null: all are there), and which row of the call each
    // is (null: the same), by which the policy's vectors, its outputs and a per-row dloss go
    const int *counting;
    const int *index;
    int loss_by_index;     // 1: loss_rows too
    float *rest;           // null, or [rows]: what rounding left of the label's entry of G
};

struct TransposeParams {
    const __nv_bfloat16 *src;   // [rows][ld_src]
    int ld_src;
    __nv_bfloat16 *dst_t;       // [cols][ld_t]
    int ld_t;
    int rows, cols;
    // rows that add nothing become zeros whatever they hold: those whose label does not count
    // (y, of the chunk's rows, or null), those whose coefficient is 0 (coef, or null)
    const long long *y;
    long long V, ignore_index;
    const float *coef;
};


// The step between a chunk's logits GEMM and its gradient GEMMs on the fused
// path, one launch: for each row, lse from the slab partials, the row's loss,
// and P' -> G in place (each of `segs` CTAs of a row recomputes the row's lse
// from the partials, in the same order, and rescales its own segment of the
// row); then, in the CTAs after those, the H chunk transposed for the dW
// contraction (tp.rows == 0: no transpose).
constexpr int PREP_THREADS = 256;
constexpr int PREP_VPT = 8;                                  // 8-column vectors per thread
constexpr int PREP_VEC_PER_CTA = PREP_THREADS * PREP_VPT;    // 2048 vectors = 16384 columns
struct PrepParams {
    MergeParams m;              // parts, zy, y, hdr, dloss, scales, lse, loss_rows
    int ldg;
    int segs;                   // CTAs per row
    TransposeParams tp;
    int tt_x;                   // transpose tiles along D (64 columns each)
};

// Cross-entropy over precomputed logits Z [N][ld] (bf16 or fp32), one row at a time.
enum : int { CE_BF16 = 0, CE_FP32 = 1, CE_FP16 = 2 };   // logits dtype codes of lce_ce_logits

struct CELogitsParams {
    const void *Z;
    void *dZ;              // null: forward only; may equal Z (gradient written in place)
    long long ld;          // row stride of Z and dZ (elements)
    int dtype;             // CE_BF16, CE_FP32 or CE_FP16
    long long N, V;
    long long ignore_index;
    const long long *y;
    int *hdr;              // workspace header: N_valid in, status flags out
    const float *dloss;
    int dloss_per_row;
    int mean;
    float *lse;            // [N]
    float *loss_rows;      // [N]
};

// Losses on answers over logits Z [N][ld] (lce_answers.cu).
struct AnswerParams {
    const void *Z;
    void *dZ;              // null: no gradient; may equal Z. Rows lie as Z's do (ld, and the address mod 16)
    long long ld;
    int dtype;             // CE_BF16, CE_FP32 or CE_FP16
    long long N, V;
    long long ignore_index;
    const long long *y;
    int *hdr;
    const float *dloss;
    int dloss_per_row, mean;
    PolicyParams pol;      // adv null: the row loss is -log p of the label, and there is no gradient
    float2 *max_sum;       // [N] or null: the row's largest logit and the sum of exp(z - it)
    float *loss_rows;      // [N]
    float *loss;           // the sum of the row losses (over N_valid where `mean`), or null
    // the gradient of a preference: row i of dZ is (p - onehot) coef[i]
    const float *coef;
};
// Pairs of sequences: the rows of sequence s are offsets[s] .. offsets[s + 1] - 1, the chosen
// one of pair k is sequence k, the rejected one sequence pairs + k.
struct PairParams {
    const long long *offsets;   // [2 pairs + 1]
    int *clean;                 // null, or [2 pairs + 1]: their running maxima, within [0, N] (launch_offsets)
    long long pairs, N, V, ignore_index;
    const long long *y;
    const float *loss_rows;     // [N]: -log p of each counting row
    const float2 *fix;          // null, or [N] (as loss_rows): what a right label logit adds to log p, and its weight
    const int *place;           // null, or where row i of the call is in loss_rows, fix and coef
    const float *ref;           // [2 pairs] or null (0)
    float beta, smoothing;
    int average;                // log probabilities per counting row
    const float *dloss;         // null, one number, or one per pair
    int dloss_per_pair, mean;
    float *seq_logp;            // [2 pairs]
    float *pair_loss;           // [pairs]
    float *loss;                // or null
    float *coef;                // [N] or null
    int *hdr;
};

// final RMSNorm (forward and backward row kernels)
constexpr int NRM_THREADS = 256;
constexpr int NRM_GRID = 256;                        // fixed: one dgamma partial slot per CTA
constexpr long long NRM_MAX_D = NRM_THREADS * 8 * 4; // 4 vectors of 8 bf16 per thread

struct NormParams {
    const __nv_bfloat16 *X;      // [rows][D]
    const __nv_bfloat16 *gamma;  // [D]
    __nv_bfloat16 *H;            // forward output [rows][D]
    float *rstd;                 // forward output [rows] or null
    const void *dH;              // backward input [rows][D], bf16 or fp32
    int dh_fp32;
    int dh_splits;               // fp32 dH: the sum of this many partial arrays,
    long long dh_split_stride;   // this many elements apart (dh_splits <= 1: one)
    __nv_bfloat16 *dX;           // backward output [rows][D]
    float *part;                 // backward: [NRM_GRID][D] dgamma partials
    int first;                   // 1: the partials start from zero
    long long rows;
    int D;
    float eps;
};

// Drawing one token per row of logits (lce_sample.cu). A null pointer: the value that
// follows for every row.
struct SampleParams {
    const void *Z;
    long long ld, N;
    int V;
    int dtype;                // CE_BF16, CE_FP32 or CE_FP16
    const float *u;           // [N]
    const float *temperature; // [N] or null
    const int *top_k;
    const float *top_p;
    const float *min_p;
    float temperature_all;
    int top_k_all;
    float top_p_all, min_p_all;
    long long *tokens;        // [N]
    float *logprobs;          // [N] or null
};
// 2^(-j / 256) in units of 2^-31; ln(2) / 256 in three parts (the last negative), its inverse
// (negative), the number that rounds to whole numbers, and the polynomial of exp
struct SampleTables {
    unsigned fix[256];
    float2 c1, c2, mc3, ninv, magic, mmagic, p3, p2, p1, round;
};
constexpr long long SMP_MAX_V = 1ll << 20;   // weights of 2^43 in 64-bit sums

// Gradient norm and clipping (lce_clip.cu).
enum : int { CLIP_NORM_2 = 0, CLIP_NORM_INF = 1, CLIP_NORM_1 = 2 };
struct ClipItem {
    const void *src;
    void *dst;             // where the scaled values go (src: in place)
    long long n;           // values
    int dtype;             // CE_BF16, CE_FP32 or CE_FP16
    long long chunks;
};
// The list as it travels in the kernels' parameters (at most 32764 bytes).
template <int CAP> struct ClipTable {
    const void *src[CAP];
    void *dst[CAP];
    long long count[CAP];  // values * 4 + dtype
    int first[CAP + 1];    // first chunk
    int n;
};
// A list of few tensors goes by a smaller table: 56 tensors of 5000 values take 7.6 us, by the large
// one, whose 29 KB of parameters go with every launch, 7.8.
constexpr int CLIP_FEW_TENSORS = 64;
constexpr int CLIP_MAX_TENSORS = 1024;   // per launch
constexpr long long CLIP_MAX_CHUNKS = 1ll << 30;   // per launch
constexpr int CLIP_MAX_PARTS = 1024;     // partial sums (CTAs) per launch
struct ClipScale {
    int kind;
    const double *part;
    int nparts;
    float max_norm, eps;
    int copy;              // 1: some destination is another place than its source
    int tell;              // 1: this launch writes the norm
    float *norm_out;
};

// 4-bit linear layers (lce_int4.cu).
struct Int4Params {
    const void *X;             // [M][ldx], bf16 or fp16
    long long ldx;
    int dtype;                 // of X, the scales and the result
    int x_vec;                 // rows of X are 16-byte aligned
    const uint8_t *q;          // [V][ldq] bytes: two values each, rows on 16 bytes
    long long ldq;
    const void *scale;         // [V][lds]
    long long lds;
    int group;                 // 32, 64 or 128 values
    int M, V, D;
    void *out;                 // [M][ldc]
    long long ldc;
    int units;                 // of 128 values (set by the launcher)
};
// The same on tcgen05: A the weight's rows, B the tokens as launch_int4_tokens lays them out.
struct Int4TileParams {
    CUtensorMap tmQ;           // [V][row bytes] packed rows, boxes of 128 bytes x 128 rows
    CUtensorMap tmX;           // [M][128 units] fp16, boxes of 64 x N
    const void *scale;         // [V][lds]
    long long lds;
    float *down;               // [M]: what a token's sums are multiplied by
    void *out;
    long long ldc;
    int dtype, M, V, D, units, groups;
    int per;                   // groups of a unit
    int row_tiles, token_tiles, stages;
    int bring;                 // 0: no stage is brought, so that every wait runs out (self-test)
    int *hdr;
    unsigned long long timeout_ns;
};
constexpr long long I4_MAX_D = 65536;   // (one token's values and a warp's buffers fit into shared memory)
struct Int4QuantParams {
    const void *W;             // [V][ldw]
    long long ldw, V;
    int D, dtype, group;
    uint8_t *q;                // [V][ldq]
    long long ldq;
    void *scale;               // [V][lds]
    long long lds;
    int scale_dtype;           // CE_BF16 or CE_FP16
};

// 8-bit linear layers (lce_fp8.cu).
struct Fp8QuantParams {
    const void *X;             // [R][ld]
    long long ld, R, C;
    long long rblocks, cblocks;   // blocks of 128
    int vec;                   // rows are 16-byte aligned
    uint8_t *q;                // [R][ldq] or null
    long long ldq;
    float *scale;              // [cblocks][R] (rows) or [rblocks][cblocks] (tiles)
    uint8_t *qt;               // X^T: [C][ldqt] or null
    long long ldqt;
    float *scale_t;            // [rblocks][C] or [cblocks][rblocks]
};
struct Fp8GemmParams {
    CUtensorMap tmA, tmB, tmC;
    int M, N, KB;              // KB: k blocks of 128
    int n_bulk;                // columns that tmC stores: N less what does not fill 16 bytes
    int m_tiles, n_tiles, tiles;
    int a_box_rows;            // rows of A's load box
    int stages;                // of the pipeline (one CTA per tile)
    int parts;                 // of k in which each tile is taken (pairs): C is then [parts][256 m_tiles][ldc]
    const float *sa;           // of A's row m and block b: sa[m * sa_row + b * sa_block]
    const float *sb;           // of B's row (or 128 rows) n and block b
    long long sa_row, sa_block, sb_row, sb_block;
    int sb_vec;                // scales of consecutive rows of B lie side by side, 16-byte aligned
    void *C;
    long long ldc;
    int c_type;                // CE_BF16, CE_FP32 or CE_FP16
    int *hdr;
    unsigned long long timeout_ns;
};

// launchers (return cudaError_t of the launch)
// cluster = 1: one CTA per 128 x 256 tile; 2: a CTA pair per 256 x 256 tile
// (tcgen05 cta_group::2, each CTA loading its own A rows and half of B).
// `grid` counts CTAs (a multiple of `cluster`).
cudaError_t launch_gemm(int mode, int cluster, const GemmParams &p, int grid, cudaStream_t s);
cudaError_t gemm_max_pairs(int *pairs);
cudaError_t launch_label_scan(const long long *y, long long N, long long V, long long ign,
                              int *hdr, cudaStream_t s);
// *out (device int64) = number of labels in [0, V) that are not ign
cudaError_t launch_count_valid(const long long *y, long long N, long long V, long long ign,
                               long long *out, cudaStream_t s);
// hdr[HDR_NVALID] = *n_total (device int64), for a mean over several shards' rows
cudaError_t launch_set_nvalid(const long long *n_total, int *hdr, cudaStream_t s);
cudaError_t launch_merge(const MergeParams &p, cudaStream_t s);
cudaError_t launch_transpose(const TransposeParams &p, cudaStream_t s);
cudaError_t launch_prep(const PrepParams &p, cudaStream_t s);
cudaError_t launch_loss_finalize(const float *loss_rows, long long N, const int *hdr,
                                 float *loss, int mean, cudaStream_t s);
// Answers over logits: the scan of the labels (which clears the header), the rows' losses (and
// the policy's gradient), the pairs, and the preference's gradient.
cudaError_t launch_answer_scan(const long long *y, long long N, long long V, long long ign, int *hdr,
                               cudaStream_t s);
cudaError_t launch_answer_rows(const AnswerParams &p, int sms, cudaStream_t s);
cudaError_t launch_answer_grad(const AnswerParams &p, int sms, cudaStream_t s);
constexpr long long PAIRS_BY_THEMSELVES = 512;   // without launch_offsets
cudaError_t launch_offsets(const PairParams &p, cudaStream_t s);
cudaError_t launch_pairs(const PairParams &p, cudaStream_t s);
// dst[i] = src[i] * *scale
cudaError_t launch_scale(const void *src, int src_dtype, const float *scale, long long n, void *dst, int dst_dtype,
                         int sms, cudaStream_t s);
cudaError_t answers_set_attributes();
cudaError_t launch_ce_logits(const CELogitsParams &p, int sms, cudaStream_t s);
cudaError_t gemm_set_attributes();
cudaError_t aux_set_attributes();
cudaError_t ce_set_attributes();
cudaError_t launch_wait_selftest(int *hdr, unsigned long long limit_ns, cudaStream_t s);
// dst[i] (bf16 / fp16, n elements) = (accumulate ? dst[i] : 0) + the sum over
// s = 0 .. splits-1, in that order, of src[s * stride + i] (fp32)
// The rows that count: index[j] = the j-th one, place[i] = where row i is among them (-1: it does not count),
// labels[j] its label (ignore_index behind the last), their number and the range check into hdr.
cudaError_t launch_compact(const long long *y, long long N, long long V, long long ign, int *hdr, int *index,
                           int *place, long long *labels, cudaStream_t s);
// dst[j][D] = src[index[row0 + j]][D] for the rows there are of [row0, row0 + rows), zeros up to a multiple of 64
// The lists of LabelRests for the chunk's labels y (counting, row0: as for the rows brought together).
cudaError_t launch_label_lists(const long long *y, const int *counting, long long row0, long long rows, long long V,
                               long long ign, int *first, int *next, int sms, int *launches, cudaStream_t s);
// What a chunk's rows are brought together from, and (W given) their labels' logits taken from.
struct GatherParams {
    const uint4 *src;            // H: the call's (with index) or the chunk's
    const int *index;            // null: the rows lie there already
    const int *counting;
    uint4 *dst;
    int row0, rows, vecs;
    const uint4 *W;              // null: no logits
    const long long *y;          // of the chunk's rows
    long long V, ignore_index;
    float inv_t;
    float *zx;
};
cudaError_t launch_gather_rows(const GatherParams &p, int sms, cudaStream_t s);
// dst[index[row0 + j]] = (accumulate ? that : 0) + the sum over s of src[s * stride + j D ..], as launch_combine_dh
cudaError_t launch_scatter_dh(const float *src, int splits, long long stride, const int *index, const int *counting,
                              long long row0, long long rows, long long D, const float *rest, const long long *y, const uint4 *W,
                              __nv_bfloat16 *dst, bool accumulate, int sms, cudaStream_t s);
cudaError_t launch_combine_dh(const float *src, int splits, long long stride, void *dst,
                              long long n, bool f16, bool accumulate, int sms, cudaStream_t s);
cudaError_t launch_rmsnorm_fwd(const NormParams &p, cudaStream_t s);
cudaError_t launch_rmsnorm_bwd(const NormParams &p, cudaStream_t s);
cudaError_t launch_dgamma_reduce(const float *part, int D, float *dgamma, cudaStream_t s);

cudaError_t sample_set_attributes();
cudaError_t launch_sample(const SampleParams &p, int sms, cudaStream_t s);
long long clip_chunks(const void *p, long long n, int dtype);
// *parts: partial sums written to `part`
cudaError_t launch_grad_norm(const ClipItem *items, int n, int kind, double *part, int sms, int *parts,
                             cudaStream_t s);
cudaError_t launch_grad_scale(const ClipItem *items, int n, const ClipScale &c, int sms, cudaStream_t s);

cudaError_t int4_set_attributes();
cudaError_t launch_int4(Int4Params p, int sms, cudaStream_t s);
bool int4_few(long long M, long long D, int group);
int int4_tile_tokens(long long M);
cudaError_t launch_int4_tokens(const Int4TileParams &p, const void *X, long long ldx, int x_vec, void *to, cudaStream_t s);
cudaError_t launch_int4_tiles(Int4TileParams p, int n, int sms, cudaStream_t s);
cudaError_t launch_int4_quantize(const Int4QuantParams &p, cudaStream_t s);

cudaError_t fp8_set_attributes();
cudaError_t launch_fp8_quantize(const Fp8QuantParams &p, int dtype, bool tile, cudaStream_t s);
// pair: CTA pairs on 256 x 256 tiles (cluster = 2); otherwise 128 x 128 tiles, each split
// along k over `cluster` CTAs (cluster > 1: one tile per cluster)
// overlap: the kernel launched just before on the stream is the quantisation of A (its
// launch may overlap this one's prologue; the kernel waits for its end)
cudaError_t launch_fp8_matmul(const Fp8GemmParams &p, bool pair, bool b_rows, int cluster, int clusters,
                              bool overlap, cudaStream_t s);
// Adds p's parts into the result.
cudaError_t launch_fp8_parts(const Fp8GemmParams &p, void *out, long long ldc, int c_type, cudaStream_t s);

constexpr float LOG2E_F = 1.4426950408889634f;

// Largest vocabulary: keeps every TMA coordinate and tile index in int32.
constexpr long long MAX_V = 1ll << 30;

}  // namespace lce
