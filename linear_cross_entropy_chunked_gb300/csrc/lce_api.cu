// C ABI of the fused chunked linear + cross-entropy library: argument checks,
// workspace layout, tensor-map encoding and the per-chunk launch sequence.
// Declarations and the contract of every entry point are in include/lce.h.
//
// The token axis is cut into chunks of `chunk` rows ("Arquitectura interna de
// Unsloth y optimizacion en Triton", section 3: token blocks; "Unsloth
// Architecture: Manual Triton Backpropagation, Fused Cross-Entropy, and 80% VRAM
// Cut", pillar 1: chunks of tokens, logits discarded after each chunk). The
// only HBM state beyond the outputs is O(chunk * V): the (max, sumexp) slab
// partials of a chunk and bf16 [chunk, V] buffers that hold exp(z - slab max),
// then G: two by default (chunks go in pairs that share one dW contraction),
// one with LCE_LOW_MEMORY.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstdlib>
#include <memory>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/lce.h"
#include "lce_internal.h"

using namespace lce;

namespace {

thread_local int g_launches = 0;

constexpr unsigned long long kDefaultTimeoutNs = 2000000000ull;  // 2 s per pipeline wait

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::mutex g_mu;
constexpr int kMaxDevices = 64;
bool g_dev_ready[kMaxDevices] = {};
int g_dev_sms[kMaxDevices] = {};
int g_dev_pairs[kMaxDevices] = {};   // co-resident CTA pairs of the GEMM kernel (0: no pairs)
bool g_dev_fp8[kMaxDevices] = {};    // the 8-bit product's kernels can run (else only its calls fail)

// GEMM tiles run on CTA pairs (tcgen05 cta_group::2, 256 x 256 tiles) when the
// device can co-schedule them; LCE_GEMM_CLUSTER=1 selects one CTA per 128 x 256
// tile instead (same work and results; measured ~8 % slower on the Llama-3 head).
int cluster_choice() {
    const char *e = getenv("LCE_GEMM_CLUSTER");
    return (e && e[0] == '1') ? 1 : 2;
}

lce_status init_device(int *sms, int *pairs) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LCE_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return LCE_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_encode) {
        cudaDriverEntryPointQueryResult q;
        void *fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn)
            return LCE_ERR_CUDA;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    if (!g_dev_ready[dev]) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return LCE_ERR_CUDA;
        if (major != 10 || minor != 3) return LCE_ERR_UNSUPPORTED;
        if (gemm_set_attributes() != cudaSuccess) return LCE_ERR_CUDA;
        if (aux_set_attributes() != cudaSuccess) return LCE_ERR_CUDA;
        if (ce_set_attributes() != cudaSuccess) return LCE_ERR_CUDA;
        if (answers_set_attributes() != cudaSuccess) return LCE_ERR_CUDA;
        if (int4_set_attributes() != cudaSuccess) return LCE_ERR_CUDA;
        if (sample_set_attributes() != cudaSuccess) return LCE_ERR_CUDA;
        g_dev_fp8[dev] = fp8_set_attributes() == cudaSuccess;
        if (!g_dev_fp8[dev]) cudaGetLastError();
        int np = 0;
        if (gemm_max_pairs(&np) != cudaSuccess) {
            cudaGetLastError();
            np = 0;
        }
        g_dev_sms[dev] = n;
        g_dev_pairs[dev] = np;
        g_dev_ready[dev] = true;
    }
    *sms = g_dev_sms[dev];
    *pairs = cluster_choice() == 2 ? g_dev_pairs[dev] : 0;
    return LCE_OK;
}

// Whether the 8-bit product's kernels can run on the current device, which init_device has set up.
bool fp8_ready() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    std::lock_guard<std::mutex> lock(g_mu);
    return g_dev_fp8[dev];
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

struct Layout {
    long long C = 0;         // rows per chunk
    long long nchunks = 0;
    int nparts = 0;          // 128-column slabs per row
    int ldg = 0;             // row stride of the chunk buffer (elements)
    int ldt = 0;             // row stride (elements) of H^T: rows of one chunk (or of a
                             // pair of chunks) rounded up to 64
    int nbuf = 1;            // chunk buffers: with two, the dW contraction of a pair of
                             // chunks runs once, over both chunks' G (K = 2 chunks)
    size_t gbuf_bytes = 0;   // bytes of one chunk buffer (the two are contiguous)
    bool frozen_w = false;   // no dW contraction (LCE_FROZEN_W)
    bool answers = false;    // a loss on answers: only some of the rows may count
    int dh_splits = 1;       // vocabulary parts of a full chunk's dH tiles
    long long ldp = 0;       // rows per fp32 dH partial array: chunk rows rounded up to 128
    size_t off_loss_rows = 0, off_zy = 0, off_parts = 0, off_G = 0, off_HT = 0, off_dHp = 0;
    size_t total = 0;
    size_t fwd_total = 0;    // the forward's share: header, row losses, target logits, partials
    size_t hdr_bytes = 0;
};

// Vocabulary parts of the dH tiles of a chunk of `rows` rows (CTA-pair tiles of
// 256 x 512): enough for DH_SPLIT_TILES tiles, at most DH_MAX_SPLITS and at most
// one per 64-column k block; one below DH_SPLIT_MIN_V. A function of the shapes
// alone, so a result does not depend on the device it ran on.
// With W frozen the dH tiles have the GPU to themselves: they are split into the
// most parts (at most DH_MAX_SPLITS) that keep them within one wave of the
// DH_ALONE_PAIRS CTA pairs a GB300 holds at once (152 SMs).
// Losses on answers, where some of the rows count and only the device knows how many: into parts for two
// waves. 1954 of 2777 rows x 50257 x 1600, all in one chunk: 617 us for the gradient in one part (32 of its 44 tiles there,
// on 76 pairs), 243 in four; 487 of 700 rows: 155 -> 97; 1071 of 1531, where one wave is nearly full: 158 -> 154. (Three
// waves: 252, 86 and 165.) With W trained too where a chunk has more than DH_BESIDE_TILES: the tiles are one long wave then that
// leaves dW little beside it and gets out of step, which reads W and G again (1843 of 2048 rows x 128256 x 4096, a whole pass:
// 3800 to 5200 us, among other work 3990 to 4430, in three parts 4030 and 4040 to 4170; 1440 rows: 3130 and 3140 to 3260, in three
// 3025 and 3120 to 3200; the spread gets narrower, its middle hardly moves). 32 tiles are what dW goes well beside (8000 rows x
// 32000 x 2048, gradients: 1340 us, in four to six parts 1400); nothing was measured between 32 and 64.
constexpr int DH_ALONE_PAIRS = 76;
constexpr int DH_BESIDE_TILES = 40;
constexpr int DH_ANSWERS_MAX_SPLITS = 16;

int dh_splits_for(long long rows, long long D, long long V, bool frozen_w = false, bool answers = false) {
    if (V < DH_SPLIT_MIN_V || rows <= 0) return 1;
    const long long tiles = cdiv(cdiv(rows, BM), 2) * cdiv(D, BN_WIDE);
    long long sp = frozen_w ? DH_ALONE_PAIRS / tiles : cdiv(DH_SPLIT_TILES, tiles);
    if (sp > DH_MAX_SPLITS) sp = DH_MAX_SPLITS;
    if (answers && (frozen_w || tiles > DH_BESIDE_TILES)) {
        sp = cdiv(2 * DH_ALONE_PAIRS, tiles);
        if (sp > DH_ANSWERS_MAX_SPLITS) sp = DH_ANSWERS_MAX_SPLITS;
    }
    if (sp > cdiv(V, BK)) sp = cdiv(V, BK);
    return sp < 1 ? 1 : static_cast<int>(sp);
}

bool make_layout(long long N, long long D, long long V, long long chunk, Layout &L,
                 bool frozen_w = false, bool low_mem = false, bool answers = false) {
    if (N < 0 || D <= 0 || V <= 0 || chunk <= 0) return false;
    if (D % 8 != 0) return false;
    if (N > 0x7fffffffll || D > 0x7fffffffll || V > MAX_V) return false;
    L.C = chunk < (N > 0 ? N : 1) ? chunk : (N > 0 ? N : 1);
    L.nchunks = N > 0 ? cdiv(N, L.C) : 0;
    L.nparts = static_cast<int>(cdiv(V, PART_COLS));
    L.ldg = static_cast<int>(align_up(static_cast<size_t>(V), BN));
    if (static_cast<unsigned long long>(L.C) * L.ldg > (1ull << 40)) return false;
    L.hdr_bytes = align_up(sizeof(int) * (HDR_COUNTERS + 3 * L.nchunks + 2), 1024);
    size_t off = L.hdr_bytes;
    L.off_loss_rows = off;
    off += align_up(sizeof(float) * static_cast<size_t>(N > 0 ? N : 1), 1024);
    L.off_zy = off;
    off += align_up(sizeof(float) * static_cast<size_t>(L.C), 1024);
    L.off_parts = off;
    off += align_up(sizeof(float2) * static_cast<size_t>(L.C) * L.nparts, 1024);
    L.off_G = off;
    L.fwd_total = off;
    // two chunk buffers when there is a dW contraction and more than one chunk:
    // chunks are taken in pairs, the second chunk's G goes into the buffer after the
    // first's, and one dW contraction runs over both (K = the pair's rows), which
    // halves the fp32 read-modify-write of dW (LCE_LOW_MEMORY: one buffer, one dW
    // contraction per chunk). The buffers are contiguous rows of one [2C][ldg]
    // array (2 * C * ldg bytes each, a multiple of 512), and the second chunk's
    // columns of H^T start at column C, which the transpose's 16-byte stores need to
    // be a multiple of 8.
    // With W frozen there is no dW contraction; two buffers then let a chunk's
    // logits GEMM run on the CTA pairs its predecessor's dH GEMM leaves free.
    L.nbuf = (!low_mem && L.nchunks > 1 && (frozen_w || L.C % 8 == 0)) ? 2 : 1;
    L.gbuf_bytes = 2 * static_cast<size_t>(L.C) * L.ldg;
    off += align_up(static_cast<size_t>(L.nbuf) * L.gbuf_bytes, 1024);
    // H chunk^T [D][ldt]: the K-major B operand of the dW contraction (none when W
    // is frozen)
    L.frozen_w = frozen_w;
    L.ldt = static_cast<int>(align_up(static_cast<size_t>(L.nbuf) * L.C, 64));
    L.off_HT = off;
    if (!frozen_w) off += align_up(2 * static_cast<size_t>(D) * L.ldt, 1024);
    // fp32 dH partial sums of a split dH contraction, one [ldp][D] array per part
    // (a single array, past `total`, serves callers that accumulate into dH)
    L.answers = answers;
    L.dh_splits = dh_splits_for(L.C, D, V, frozen_w, answers);
    // the first chunk of a pair runs its dH tiles alone (split for all pairs)
    if (L.nbuf == 2 && dh_splits_for(L.C, D, V, true) > L.dh_splits)
        L.dh_splits = dh_splits_for(L.C, D, V, true);
    L.ldp = static_cast<long long>(align_up(static_cast<size_t>(L.C), BM));
    L.off_dHp = off;
    if (L.dh_splits > 1)
        off += align_up(4 * static_cast<size_t>(L.dh_splits) * L.ldp * static_cast<size_t>(D), 1024);
    L.total = off;
    return true;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Workspace of the final-RMSNorm path: the loss path's layout, then the chunk's
// normalised rows H (bf16), the chunk's dH (fp32) and the dgamma partials.
struct NormLayout {
    Layout L;
    size_t off_H = 0, off_dH = 0, off_part = 0, total = 0;
};

// Bytes past the loss path's workspace that accumulating into dH (and the
// RMSNorm path) need: one fp32 dH array for the chunk, added to the caller's dH
// once the chunk is done; none when the layout already holds split partials.
size_t acc_dh_bytes(const Layout &L, long long D) {
    if (L.dh_splits > 1) return 0;
    return align_up(4 * static_cast<size_t>(L.ldp) * static_cast<size_t>(D), 1024);
}

bool make_norm_layout(long long N, long long D, long long V, long long chunk, NormLayout &NL,
                      bool frozen_w = false, bool low_mem = false) {
    // W trained: chunk pairs with one dW contraction each, as on the loss path; W
    // frozen: one chunk buffer
    if (!make_layout(N, D, V, chunk, NL.L, frozen_w, low_mem || frozen_w)) return false;
    if (D > NRM_MAX_D) return false;
    // the chunk's dH (fp32): the layout's partial arrays, or one array past them
    NL.off_dH = NL.L.off_dHp;
    size_t off = NL.L.total + acc_dh_bytes(NL.L, D);
    NL.off_H = off;   // the normalised rows of a chunk (of a pair of chunks with two buffers)
    off += align_up(2 * static_cast<size_t>(NL.L.nbuf) * NL.L.C * D, 1024);
    NL.off_part = off;
    off += align_up(4 * static_cast<size_t>(NRM_GRID) * D, 1024);
    NL.total = off;
    return true;
}

// Element types of the tensor maps.
enum MapType { MAP_BF16, MAP_F16, MAP_F32, MAP_U8 };

// Tensor map over a row-major array with the 128-byte swizzle of the MMA
// operand tiles and of the epilogue staging boxes; zero fill out of bounds on
// loads, clipping on stores.
bool encode_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims,
                const uint64_t *strides_bytes, const uint32_t *box, MapType type) {
    cuuint64_t d[3];
    cuuint64_t st[2];
    cuuint32_t bx[3];
    cuuint32_t es[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        bx[i] = box[i];
    }
    for (int i = 0; i + 1 < rank; ++i) st[i] = strides_bytes[i];
    const CUtensorMapDataType dt = type == MAP_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : type == MAP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                   : type == MAP_U8  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUresult r = g_encode(m, dt,
                          rank, const_cast<void *>(base), d, st, bx, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// MMA operand tile load map: 2-D, 16-bit (bf16 or fp16) or 8-bit elements, box
// {box_inner, box_outer}.
bool encode_2d(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer,
               uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
               MapType type = MAP_BF16) {
    const uint64_t dims[2] = {inner, outer};
    const uint64_t st[1] = {row_stride_bytes};
    const uint32_t box[2] = {box_inner, box_outer};
    return encode_map(m, base, 2, dims, st, box, type);
}

// Epilogue store map: 2-D, box = 128 bytes x box_rows rows (128: a column half
// of a gradient tile; 32: one warp's rows of a logits tile).
bool encode_store_2d(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer,
                     uint64_t row_stride_bytes, MapType type, uint32_t box_rows = 128) {
    const uint64_t dims[2] = {inner, outer};
    const uint64_t st[1] = {row_stride_bytes};
    const uint32_t box[2] = {type == MAP_F32 ? 32u : 64u, box_rows};
    return encode_map(m, base, 2, dims, st, box, type);
}

struct Ctx {
    const __nv_bfloat16 *H, *W;
    const long long *y;
    long long N, D, V, ign;
    Layout L;
    uint8_t *ws;
    int *hdr;
    float *loss_rows, *zy;
    float *zx = nullptr;         // [C]: the labels' logits as dot products of their own (the preference loss),
    float2 *fix = nullptr;       // [N]: what the log probabilities move by with them
    float2 *parts;
    __nv_bfloat16 *Gb[2];   // the chunk buffers (Gb[1] == Gb[0] with one)
    __nv_bfloat16 *HT;
    int sms;
    int pairs;   // > 0: GEMMs run as CTA pairs (cluster of 2), at most this many at once
    int reduction;       // LCE_REDUCTION_*
    bool h_chunked;      // H is a buffer of one chunk's rows (of a pair's with two chunk
                         // buffers: chunk k at rows (k mod 2) * C), refilled per chunk
    bool f16;            // H, W, G and dH are fp16 (bf16 otherwise)
    MapType t16;         // the 16-bit map type of this call
    cudaStream_t s;
    CUtensorMap tmH_K, tmW_K, tmW_MN;
    // losses on answers: the policy (pol.adv) and its temperature, or the rows' coefficients of a
    // preference; what a row that adds nothing holds then reaches no gradient
    PolicyParams pol{};
    float inv_t = 1.f;
    bool answers = false;
    const float *coef = nullptr;
    // the rows that count brought together, chunk by chunk into H's buffer (h_chunked): which rows of the
    // call they are (null: not done), and where H lies
    const int *index = nullptr;
    const __nv_bfloat16 *Hrows = nullptr;
    bool loss_by_index = false;
    LabelRests rests{};          // (losses on answers with gradients)
    bool dw16 = false;           // dW is bf16 (one contraction)
};

// Row of H (c.H) where the chunk starting at row0 begins.
inline long long h_row(const Ctx &c, long long row0) {
    return c.h_chunked ? ((row0 / c.L.C) % c.L.nbuf) * c.L.C : row0;
}

// ---- optional per-kernel event timing (lce_profile_*)
struct ProfPair {
    int kind;
    cudaEvent_t a, b;
};
std::mutex g_prof_mu;
std::atomic<bool> g_prof_on{false};   // read without the mutex on every launch
std::vector<ProfPair> g_prof_pending;
std::vector<cudaEvent_t> g_prof_pool;
double g_prof_ms[LCE_KERNEL_KINDS] = {};
int64_t g_prof_n[LCE_KERNEL_KINDS] = {};

cudaEvent_t prof_event() {
    if (!g_prof_pool.empty()) {
        cudaEvent_t e = g_prof_pool.back();
        g_prof_pool.pop_back();
        return e;
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
    return e;
}

// Records the start event of a launch of `kind`; returns the pair index or -1.
int prof_begin(int kind, cudaStream_t s) {
    if (!g_prof_on) return -1;
    std::lock_guard<std::mutex> lock(g_prof_mu);
    ProfPair p{kind, prof_event(), prof_event()};
    if (!p.a || !p.b) return -1;
    cudaEventRecord(p.a, s);
    g_prof_pending.push_back(p);
    return static_cast<int>(g_prof_pending.size()) - 1;
}

void prof_end(int idx, cudaStream_t s) {
    if (idx < 0) return;
    std::lock_guard<std::mutex> lock(g_prof_mu);
    cudaEventRecord(g_prof_pending[idx].b, s);
}

#define LCE_LAUNCH_KIND(kind, stream, expr)                 \
    do {                                                    \
        const int _pi = prof_begin((kind), (stream));       \
        if ((expr) != cudaSuccess) return LCE_ERR_CUDA;     \
        prof_end(_pi, (stream));                            \
        ++g_launches;                                       \
    } while (0)

#define LCE_LAUNCH(expr) LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, c.s, expr)

// A second stream per device for the dW kernel that runs beside the dH kernel
// of a gradient phase (forked from and joined back to the caller's stream
// through two events). The mutex keeps the record / wait / launch sequence of
// one call together when several host threads use the same device.
struct SideStream {
    cudaStream_t s = nullptr;
    cudaEvent_t fork = nullptr, join = nullptr;
    std::mutex mu;
};
SideStream g_side[64];
std::mutex g_side_mu;

SideStream *side_stream() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(g_side_mu);
    SideStream &ss = g_side[dev];
    if (!ss.s) {
        cudaStream_t st = nullptr;
        if (cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking) != cudaSuccess) return nullptr;
        if (cudaEventCreateWithFlags(&ss.fork, cudaEventDisableTiming) != cudaSuccess ||
            cudaEventCreateWithFlags(&ss.join, cudaEventDisableTiming) != cudaSuccess)
            return nullptr;
        ss.s = st;   // last: marks the set as complete
    }
    return &ss;
}

lce_status setup(Ctx &c, const void *H, const void *W, const int64_t *y, int64_t N, int64_t D,
                 int64_t V, int64_t ign, int64_t chunk, void *ws, size_t ws_bytes,
                 lce_stream_t stream, bool h_chunked = false, bool f16 = false,
                 bool frozen_w = false, bool fwd_only = false, bool low_mem = false,
                 bool scan = true, bool answers = false) {
    g_launches = 0;
    if (!make_layout(N, D, V, chunk, c.L, frozen_w, low_mem, answers)) return LCE_ERR_INVALID_ARG;
    if (!ws) return LCE_ERR_INVALID_ARG;
    if (N > 0 && (!H || !y)) return LCE_ERR_INVALID_ARG;
    if (!W) return LCE_ERR_INVALID_ARG;
    if (!aligned16(ws) || !aligned16(W) || (H && !aligned16(H)) || (y && !aligned16(y)))
        return LCE_ERR_ALIGNMENT;
    if (ws_bytes < (fwd_only ? c.L.fwd_total : c.L.total)) return LCE_ERR_WORKSPACE;
    lce_status st = init_device(&c.sms, &c.pairs);
    if (st != LCE_OK) return st;
    c.H = static_cast<const __nv_bfloat16 *>(H);
    c.W = static_cast<const __nv_bfloat16 *>(W);
    c.y = reinterpret_cast<const long long *>(y);
    c.N = N;
    c.D = D;
    c.V = V;
    c.ign = ign;
    c.ws = static_cast<uint8_t *>(ws);
    c.hdr = reinterpret_cast<int *>(c.ws);
    c.loss_rows = reinterpret_cast<float *>(c.ws + c.L.off_loss_rows);
    c.zy = reinterpret_cast<float *>(c.ws + c.L.off_zy);
    c.parts = reinterpret_cast<float2 *>(c.ws + c.L.off_parts);
    c.Gb[0] = reinterpret_cast<__nv_bfloat16 *>(c.ws + c.L.off_G);
    c.Gb[1] = reinterpret_cast<__nv_bfloat16 *>(c.ws + c.L.off_G +
                                                (c.L.nbuf > 1 ? c.L.gbuf_bytes : 0));
    // (with two buffers Gb[1] is row C of one [2C][ldg] array starting at Gb[0])
    c.HT = reinterpret_cast<__nv_bfloat16 *>(c.ws + c.L.off_HT);
    c.s = reinterpret_cast<cudaStream_t>(stream);
    c.reduction = LCE_REDUCTION_MEAN;
    c.h_chunked = h_chunked;
    c.f16 = f16;
    c.t16 = f16 ? MAP_F16 : MAP_BF16;
    // with CTA pairs each CTA loads its own half (128 rows) of a 256-row W tile; the
    // pair MMA reads both CTAs' halves from their shared memory
    if (!encode_2d(&c.tmW_K, W, D, V, D * 2, BK, c.pairs > 0 ? BN / 2 : BN, c.t16)) return LCE_ERR_CUDA;
    if (!encode_2d(&c.tmW_MN, W, D, V, D * 2, 64, BK, c.t16)) return LCE_ERR_CUDA;
    if (N > 0 && !encode_2d(&c.tmH_K, H, D, h_chunked ? c.L.C * c.L.nbuf : N, D * 2, BK, BM, c.t16))
        return LCE_ERR_CUDA;
    if (cudaMemsetAsync(c.ws, 0, c.L.hdr_bytes, c.s) != cudaSuccess) return LCE_ERR_CUDA;
    if (scan) LCE_LAUNCH(launch_label_scan(c.y, N, V, ign, c.hdr, c.s));
    return LCE_OK;
}

void base_params(const Ctx &c, GemmParams &p, long long row0, long long rows, int slot) {
    p.rows = static_cast<int>(rows);
    p.row0 = static_cast<int>(row0);
    p.V = static_cast<int>(c.V);
    p.D = static_cast<int>(c.D);
    p.ignore_index = c.ign;
    p.y = c.y;
    p.tile_counter = c.hdr + HDR_COUNTERS + slot;
    p.hdr = c.hdr;
    p.parts = c.parts;
    p.nparts = c.L.nparts;
    p.zy = c.zy;
    p.G = c.Gb[0];
    p.ldg = c.L.ldg;
    p.timeout_ns = kDefaultTimeoutNs;
    p.dloss_per_row = c.reduction == LCE_REDUCTION_NONE ? 1 : 0;
    p.mean = c.reduction == LCE_REDUCTION_MEAN ? 1 : 0;
    p.f16 = c.f16 ? 1 : 0;
    p.answers = c.answers ? 1 : 0;
    p.inv_t = c.inv_t;
    p.rests = c.rests;
    p.Hc = reinterpret_cast<const uint4 *>(c.H + h_row(c, row0) * c.D);
    p.W = reinterpret_cast<const uint4 *>(c.W);
    p.counting = c.index ? c.hdr + HDR_NVALID : nullptr;
}

// The logits launches of the chunk at row0 (MODE_LSE / _LSE_P / _G epilogue, P' or G
// into chunk buffer G).
struct LogitsSpec {
    int mode;
    long long row0, rows;
    int slot;
    const float *lse;       // MODE_G
    const float *dloss;
    __nv_bfloat16 *G;
};

lce_status logits_params(const Ctx &c, const LogitsSpec &l, GemmParams &p) {
    memset(&p, 0, sizeof(p));
    base_params(c, p, l.row0, l.rows, l.slot);
    p.tmA0 = c.tmH_K;
    p.a_row0 = static_cast<int>(h_row(c, l.row0));
    p.tmB0 = c.tmW_K;
    p.m_blocks0 = static_cast<int>(cdiv(l.rows, BM));
    p.n_blocks0 = static_cast<int>(cdiv(c.V, BN));
    p.k_blocks0 = static_cast<int>(cdiv(c.D, BK));
    const int cl = c.pairs > 0 ? 2 : 1;
    p.total_tiles = static_cast<int>(cdiv(p.m_blocks0, cl)) * p.n_blocks0;
    p.lse = l.lse;
    p.dloss = l.dloss;
    p.G = l.G;
    if (l.mode != MODE_LSE &&
        !encode_store_2d(&p.tmS0, l.G, c.V, l.rows, 2ull * c.L.ldg, c.t16, 32))
        return LCE_ERR_CUDA;
    return LCE_OK;
}

lce_status run_logits(const Ctx &c, int mode, long long row0, long long rows, int slot,
                      const float *lse, const float *dloss, __nv_bfloat16 *G) {
    GemmParams p;
    const lce_status st = logits_params(c, LogitsSpec{mode, row0, rows, slot, lse, dloss, G}, p);
    if (st != LCE_OK) return st;
    const int cl = c.pairs > 0 ? 2 : 1;
    const int units = cl == 2 ? c.pairs : c.sms;
    const int grid = cl * (p.total_tiles < units ? p.total_tiles : units);
    LCE_LAUNCH_KIND(LCE_KERNEL_LOGITS, c.s, launch_gemm(mode, cl, p, grid, c.s));
    return LCE_OK;
}

#define LCE_TRY(expr)                         \
    do {                                      \
        lce_status _st = (expr);              \
        if (_st != LCE_OK) return _st;        \
    } while (0)

// Where a gradient phase leaves dH: the caller's rows (bf16 / fp16, stored by the
// dH tiles directly), or fp32 partial sums, `parts` arrays of ldp rows x D (one
// per vocabulary part of the dH tiles), for a combining kernel to add up.
struct DhOut {
    void *ptr;
    bool fp32;
    int parts;
    long long ldp;
};

// Vocabulary parts for a chunk of `rows` rows: one off the CTA-pair path (its
// 256-column dH tiles are many), else the shapes' split, at most the layout's.
// alone: the dH tiles have the GPU to themselves (no dW tiles beside them).
int dh_parts(const Ctx &c, long long rows, bool alone) {
    if (c.pairs <= 0) return 1;
    const int sp = dh_splits_for(rows, c.D, c.V, c.L.frozen_w || alone, c.L.answers);
    return sp < c.L.dh_splits ? sp : c.L.dh_splits;
}

// Which rows of the chunk at row0 the transpose leaves out.
void set_row_filter(const Ctx &c, long long row0, TransposeParams &tp) {
    tp.y = c.answers && !c.coef ? c.y + row0 : nullptr;
    tp.V = c.V;
    tp.ignore_index = c.ign;
    tp.coef = c.coef ? c.coef + row0 : nullptr;
}

// H chunk^T into columns col0 .. col0 + rows - 1 of H^T (the K-major B operand of
// the dW tiles; col0 = C for the second chunk of a pair).
lce_status run_transpose(const Ctx &c, long long row0, long long rows, long long col0) {
    const __nv_bfloat16 *Hc = c.H + h_row(c, row0) * c.D;
    TransposeParams tp;
    tp.src = Hc;
    tp.ld_src = static_cast<int>(c.D);
    tp.dst_t = c.HT + col0;
    tp.ld_t = c.L.ldt;
    tp.rows = static_cast<int>(rows);
    tp.cols = static_cast<int>(c.D);
    set_row_filter(c, row0, tp);
    LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, c.s, launch_transpose(tp, c.s));
    return LCE_OK;
}

// What one gradient launch set computes. The dH tiles of the chunk at row0 read
// its G (buffer G); the dW tiles, when there are any (dw_rows > 0), contract over
// dw_rows rows of G starting at Gdw (the chunk's own rows, or the rows of a pair of
// chunks) against as many columns of H^T.
struct GradSpec {
    __nv_bfloat16 *G;
    __nv_bfloat16 *Gdw;
    long long dw_rows;      // K of the dW tiles (0: no dW tiles)
    bool transposed;        // H^T is in place (else it is made first, for this chunk)
    bool dh_alone;          // no dW tiles beside the dH tiles: split for all CTA pairs
    bool dw_only;           // the dW tiles alone (the chunk's dH is computed elsewhere)
    const LogitsSpec *beside = nullptr;   // with dh_alone: another chunk's logits tiles on
                                          // the pairs the dH tiles leave free, then on all
};

// *parts_used: the number of non-empty vocabulary parts written (fp32 output).
lce_status run_bwd(const Ctx &c, long long row0, long long rows, int slot, const DhOut &o,
                   float *dW, bool accumulate, const float *dloss, const GradSpec &g,
                   int *parts_used = nullptr) {
    GemmParams p;
    memset(&p, 0, sizeof(p));
    base_params(c, p, row0, rows, slot);
    p.dw_rows = static_cast<int>(g.dw_rows);
    p.dw_row0 = static_cast<int>(row0 + rows - g.dw_rows);
    p.G = g.G;
    void *dHc = o.ptr;
    const bool dh_fp32 = o.fp32;
    const int want_parts = (o.fp32 && o.parts > 1 && c.pairs > 0) ? o.parts : 1;
    // frozen W or the first chunk of a pair: the dH tiles only (no dW maps, dW untouched)
    const bool with_dw = !c.L.frozen_w && g.dw_rows > 0;
    const int cl = c.pairs > 0 ? 2 : 1;
    if (with_dw) {
        // the H chunk^T for the K-major B operand of the dW tiles
        if (!g.transposed) LCE_TRY(run_transpose(c, row0, rows, 0));
        // dW A = G^T read from G itself, MN-major: per k block a CTA's 128 vocabulary
        // columns x 64 rows as two 64-column blocks, fetched by one 3-D box {64
        // columns, 64 rows, 2 blocks} (x: the column within a block, y: the row, z: the
        // 64-column block, 128 bytes apart). The columns of the last block past V read
        // the buffer's padding; they meet only dW rows past V, which the store clips.
        const uint64_t dims[3] = {64, static_cast<uint64_t>(g.dw_rows),
                                  static_cast<uint64_t>(cdiv(c.V, 64))};
        const uint64_t strides[2] = {2ull * c.L.ldg, 128};
        const uint32_t box[3] = {64, BK, 2};
        if (!encode_map(&p.tmA1, g.Gdw, 3, dims, strides, box, c.t16)) return LCE_ERR_CUDA;
        if (!encode_2d(&p.tmB1, c.HT, g.dw_rows, c.D, 2ull * c.L.ldt, BK, BN / cl, c.t16))
            return LCE_ERR_CUDA;
        if (!encode_store_2d(&p.tmS1, dW, c.D, c.V, (c.dw16 ? 2ull : 4ull) * c.D, c.dw16 ? MAP_BF16 : MAP_F32))
            return LCE_ERR_CUDA;
    }
    if (!encode_2d(&p.tmA0, g.G, c.V, rows, 2ull * c.L.ldg, BK, BM, c.t16)) return LCE_ERR_CUDA;
    p.tmB0 = c.tmW_MN;
    const uint64_t s0_rows = want_parts > 1 ? static_cast<uint64_t>(want_parts) * o.ldp : rows;
    if (!encode_store_2d(&p.tmS0, dHc, c.D, s0_rows, (dh_fp32 ? 4ull : 2ull) * c.D,
                         dh_fp32 ? MAP_F32 : c.t16))
        return LCE_ERR_CUDA;
    p.m_blocks0 = static_cast<int>(cdiv(rows, BM));
    p.n_blocks0 = static_cast<int>(cdiv(c.D, BN));
    p.k_blocks0 = static_cast<int>(cdiv(c.V, BK));
    p.m_blocks1 = with_dw ? static_cast<int>(cdiv(c.V, BM)) : 0;
    p.n_blocks1 = with_dw ? static_cast<int>(cdiv(c.D, BN)) : 0;
    p.k_blocks1 = with_dw ? static_cast<int>(cdiv(g.dw_rows, BK)) : 0;
    p.total_tiles = static_cast<int>(cdiv(p.m_blocks0, cl)) * p.n_blocks0 +
                    static_cast<int>(cdiv(p.m_blocks1, cl)) * p.n_blocks1;
    int parts = 1;
    if (want_parts > 1) {
        p.kb_per_split = static_cast<int>(cdiv(p.k_blocks0, want_parts));
        parts = static_cast<int>(cdiv(p.k_blocks0, p.kb_per_split));
        p.k_splits = parts;
        p.split_rows = static_cast<int>(o.ldp);
    }
    if (parts_used) *parts_used = parts;
    p.dH = static_cast<__nv_bfloat16 *>(dHc);
    p.dh_fp32 = dh_fp32 ? 1 : 0;
    p.dloss = dloss;   // fp16: the epilogues apply the uniform part of the scale
    p.dW = dW;
    p.dw_accumulate = accumulate ? 1 : 0;
    p.dw_16 = c.dw16 ? 1 : 0;
    const int units = cl == 2 ? c.pairs : c.sms;
    // profiling kind: a pair's second chunk (its dH with both chunks' dW), a pair's
    // first chunk (its dH alone), or a chunk's whole gradient phase
    const int kind = (with_dw && g.dw_rows > rows) ? LCE_KERNEL_PHASE
                     : (!with_dw && (!c.L.frozen_w || g.beside)) ? LCE_KERNEL_DH
                                                                 : LCE_KERNEL_GRAD;
    if (cl == 2) {
        // CTA pairs: the dH tiles run 512 columns wide (two MMAs share each A
        // block: a quarter fewer operand bytes per flop) in one kernel with one
        // pair per tile (at most all pairs); the dW tiles run beside it in a
        // second kernel on the side stream, sized to exactly the pairs the dH
        // kernel leaves free, so the two grids fit on the GPU together whichever
        // the hardware dispatches first (nothing orders two ready grids on
        // separate hardware queues; a dW grid that took every SM would leave the
        // long dH tiles to run after it). A third launch, a dW grid as large as
        // the dH one, queued on the caller's stream behind the dH kernel, takes
        // over the dH kernel's SMs when it ends; both dW grids draw tiles from
        // the same counter.
        GemmParams ph = p;
        ph.n_blocks0 = static_cast<int>(cdiv(c.D, BN_WIDE));
        ph.m_blocks1 = ph.n_blocks1 = ph.k_blocks1 = 0;
        ph.total_tiles = g.dw_only ? 0 : static_cast<int>(cdiv(p.m_blocks0, cl)) * ph.n_blocks0 * parts;
        if (!with_dw && !g.beside) {
            const int gh = cl * (ph.total_tiles < units ? ph.total_tiles : units);
            if (ph.total_tiles > 0)
                LCE_LAUNCH_KIND(kind, c.s, launch_gemm(MODE_DH, cl, ph, gh, c.s));
            return LCE_OK;
        }
        if (!with_dw) {
            // the dH tiles beside another chunk's logits tiles: as with the dW grids
            // below, one logits grid on the side stream sized to the pairs the dH grid
            // leaves free and one behind the dH kernel, drawing from one counter
            GemmParams pl;
            LCE_TRY(logits_params(c, *g.beside, pl));
            SideStream *ss = side_stream();
            if (!ss) return LCE_ERR_CUDA;
            std::lock_guard<std::mutex> lock(ss->mu);
            const int dh_pairs = ph.total_tiles < units ? ph.total_tiles : units;
            const int free_pairs = units - dh_pairs;
            const int l1 = pl.total_tiles < free_pairs ? pl.total_tiles : free_pairs;
            const int l2 = pl.total_tiles < dh_pairs ? pl.total_tiles : dh_pairs;
            const int pi = prof_begin(kind, c.s);
            if (cudaEventRecord(ss->fork, c.s) != cudaSuccess ||
                cudaStreamWaitEvent(ss->s, ss->fork, 0) != cudaSuccess)
                return LCE_ERR_CUDA;
            int launched = 0;
            if (dh_pairs > 0) {
                if (launch_gemm(MODE_DH, cl, ph, cl * dh_pairs, c.s) != cudaSuccess) return LCE_ERR_CUDA;
                ++launched;
            }
            if (l1 > 0) {
                if (launch_gemm(g.beside->mode, cl, pl, cl * l1, ss->s) != cudaSuccess)
                    return LCE_ERR_CUDA;
                ++launched;
            }
            if (l2 > 0 && (dh_pairs > 0 || l1 == 0)) {
                if (launch_gemm(g.beside->mode, cl, pl, cl * l2, c.s) != cudaSuccess)
                    return LCE_ERR_CUDA;
                ++launched;
            }
            if (cudaEventRecord(ss->join, ss->s) != cudaSuccess ||
                cudaStreamWaitEvent(c.s, ss->join, 0) != cudaSuccess)
                return LCE_ERR_CUDA;
            prof_end(pi, c.s);
            g_launches += launched;
            return LCE_OK;
        }
        GemmParams pw = p;
        pw.m_blocks0 = 0;
        pw.k_splits = 0;
        pw.total_tiles = static_cast<int>(cdiv(p.m_blocks1, cl)) * p.n_blocks1;
        pw.tile_counter = c.hdr + HDR_COUNTERS + 2 * c.L.nchunks + 2 + slot / 2;
        SideStream *ss = side_stream();
        if (!ss) return LCE_ERR_CUDA;
        std::lock_guard<std::mutex> lock(ss->mu);
        const int dh_pairs = ph.total_tiles < units ? ph.total_tiles : units;
        const int free_pairs = units - dh_pairs;
        const int w1 = pw.total_tiles < free_pairs ? pw.total_tiles : free_pairs;
        const int w2 = pw.total_tiles < dh_pairs ? pw.total_tiles : dh_pairs;
        const int pi = prof_begin(kind, c.s);
        if (cudaEventRecord(ss->fork, c.s) != cudaSuccess ||
            cudaStreamWaitEvent(ss->s, ss->fork, 0) != cudaSuccess)
            return LCE_ERR_CUDA;
        int launched = 0;
        if (dh_pairs > 0) {
            if (launch_gemm(MODE_DH, cl, ph, cl * dh_pairs, c.s) != cudaSuccess) return LCE_ERR_CUDA;
            ++launched;
        }
        if (w1 > 0) {
            if (launch_gemm(MODE_BWD, cl, pw, cl * w1, ss->s) != cudaSuccess) return LCE_ERR_CUDA;
            ++launched;
        }
        if (w2 > 0 && (dh_pairs > 0 || w1 == 0)) {
            if (launch_gemm(MODE_BWD, cl, pw, cl * w2, c.s) != cudaSuccess) return LCE_ERR_CUDA;
            ++launched;
        }
        if (cudaEventRecord(ss->join, ss->s) != cudaSuccess ||
            cudaStreamWaitEvent(c.s, ss->join, 0) != cudaSuccess)
            return LCE_ERR_CUDA;
        prof_end(pi, c.s);
        g_launches += launched;
        return LCE_OK;
    }
    const int grid = cl * (p.total_tiles < units ? p.total_tiles : units);
    LCE_LAUNCH_KIND(kind, c.s, launch_gemm(MODE_BWD, cl, p, grid, c.s));
    return LCE_OK;
}

// A chunk's gradient launches on the loss path: dH straight into the caller's
// rows when there is one vocabulary part and nothing to accumulate, else through
// the fp32 partial arrays and the combining kernel (which adds into the caller's
// dH when accumulating).
lce_status run_grad(const Ctx &c, long long row0, long long rows, int slot, void *dHc,
                    bool acc_dh, float *dW, bool acc_dw, const float *dloss, const GradSpec &g) {
    if (g.dw_only) return run_bwd(c, row0, rows, slot, DhOut{dHc, false, 1, 0}, dW, acc_dw, dloss, g);
    if (c.rests.first) {
        int n = 1;
        LCE_LAUNCH(launch_label_lists(reinterpret_cast<const long long *>(c.y) + row0, c.index ? c.hdr + HDR_NVALID : nullptr,
                                      row0, rows, c.V, c.ign, c.rests.first, c.rests.next, c.sms, &n, c.s));
        g_launches += n - 1;
    }
    const int want = dh_parts(c, rows, g.dh_alone);
    if (want <= 1 && !acc_dh && !c.index)
        return run_bwd(c, row0, rows, slot, DhOut{dHc, false, 1, 0}, dW, acc_dw, dloss, g);
    float *dHp = reinterpret_cast<float *>(c.ws + c.L.off_dHp);
    int parts = 1;
    LCE_TRY(run_bwd(c, row0, rows, slot, DhOut{dHp, true, want, c.L.ldp}, dW, acc_dw, dloss, g,
                    &parts));
    if (c.index) {
        LCE_LAUNCH(launch_scatter_dh(dHp, parts, c.L.ldp * c.D, c.index, c.hdr + HDR_NVALID, row0, rows, c.D,
                                     c.rests.rest, reinterpret_cast<const long long *>(c.y) + row0,
                                     reinterpret_cast<const uint4 *>(c.W), static_cast<__nv_bfloat16 *>(dHc) - row0 * c.D, acc_dh, c.sms, c.s));
        return LCE_OK;
    }
    LCE_LAUNCH(launch_combine_dh(dHp, parts, c.L.ldp * c.D, dHc, rows * c.D, c.f16, acc_dh,
                                 c.sms, c.s));
    return LCE_OK;
}

void merge_params(const Ctx &c, long long row0, long long rows, float *lse, const float *dloss,
                  float *loss_rows, MergeParams &m) {
    m.parts = c.parts;
    m.nparts = c.L.nparts;
    m.inv_t = c.inv_t;
    m.zy = c.zy;
    m.zx = c.coef ? nullptr : c.zx;   // (with the coefficients the sequences have been added up)
    m.fix = c.fix;
    m.G = c.Gb[0];
    m.ldg = c.L.ldg;
    m.rows = static_cast<int>(rows);
    m.row0 = static_cast<int>(row0);
    m.V = static_cast<int>(c.V);
    m.ignore_index = c.ign;
    m.y = c.y;
    m.hdr = c.hdr;
    m.dloss = dloss;
    m.dloss_per_row = c.reduction == LCE_REDUCTION_NONE ? 1 : 0;
    m.mean = c.reduction == LCE_REDUCTION_MEAN ? 1 : 0;
    m.f16 = c.f16 ? 1 : 0;
    m.lse = lse;
    m.loss_rows = loss_rows;
    m.pol = c.pol;
    m.answers = c.answers ? 1 : 0;
    m.counting = c.index ? c.hdr + HDR_NVALID : nullptr;
    m.index = c.pol.adv ? c.index : nullptr;   // (a preference's rows go by their place)
    m.loss_by_index = c.loss_by_index ? 1 : 0;
    m.rest = c.rests.rest;
}

lce_status run_merge(const Ctx &c, long long row0, long long rows, float *lse,
                     const float *dloss, float *loss_rows) {
    MergeParams m;
    merge_params(c, row0, rows, lse, dloss, loss_rows, m);
    LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, c.s, launch_merge(m, c.s));
    return LCE_OK;
}

// Fused path, between a chunk's logits GEMM and its gradient GEMMs, one launch:
// lse and the row losses, P' -> G in place in chunk buffer G, and (transpose) the
// H chunk^T the dW tiles read, into columns ht_col0 .. of H^T.
lce_status run_prep(const Ctx &c, long long row0, long long rows, float *lse,
                    const float *dloss, float *loss_rows, __nv_bfloat16 *G, bool transpose,
                    long long ht_col0 = 0) {
    PrepParams pp;
    memset(&pp, 0, sizeof(pp));
    merge_params(c, row0, rows, lse, dloss, loss_rows, pp.m);
    pp.m.G = G;
    pp.ldg = c.L.ldg;
    pp.segs = static_cast<int>(cdiv(cdiv(c.V, 8), PREP_VEC_PER_CTA));
    if (transpose) {
        pp.tp.src = c.H + h_row(c, row0) * c.D;
        pp.tp.ld_src = static_cast<int>(c.D);
        pp.tp.dst_t = c.HT + ht_col0;
        pp.tp.ld_t = c.L.ldt;
        pp.tp.rows = static_cast<int>(rows);
        pp.tp.cols = static_cast<int>(c.D);
        set_row_filter(c, row0, pp.tp);
        pp.tt_x = static_cast<int>(cdiv(c.D, 64));
    }
    LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, c.s, launch_prep(pp, c.s));
    return LCE_OK;
}

// Rows of chunk k (the last chunk may be shorter).
inline long long chunk_rows(const Ctx &c, long long k) {
    const long long row0 = k * c.L.C;
    return (c.N - row0) < c.L.C ? (c.N - row0) : c.L.C;
}

// Whether chunks are taken in pairs with one dW contraction per pair: CTA pairs,
// a dW contraction, two chunk buffers (so more than one chunk), H in place.
inline bool paired(const Ctx &c, bool h_chunked_ok = false) {
    return c.pairs > 0 && !c.L.frozen_w && c.L.nbuf == 2 && (h_chunked_ok || !c.h_chunked);
}

// W frozen with two chunk buffers: chunk k+1's logits tiles run on the CTA pairs
// chunk k's dH tiles leave free (chunk k in buffer k % 2).
inline bool frozen_overlapped(const Ctx &c) {
    return c.pairs > 0 && c.L.frozen_w && c.L.nbuf == 2 && !c.h_chunked;
}

// The rows of chunk k that count into their place of H's buffer (nothing to do where H is read in place), and
// with_labels their labels' logits.
lce_status bring_rows(const Ctx &c, long long k, bool with_labels) {
    if (!c.index && !with_labels) return LCE_OK;
    const long long row0 = k * c.L.C;
    const __nv_bfloat16 *Hc = c.H + h_row(c, row0) * c.D;
    GatherParams p;
    p.src = reinterpret_cast<const uint4 *>(c.index ? c.Hrows : Hc);
    p.index = c.index;
    p.counting = c.index ? c.hdr + HDR_NVALID : nullptr;
    p.dst = reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(Hc));   // (written with an index only)
    p.row0 = static_cast<int>(row0);
    p.rows = static_cast<int>(chunk_rows(c, k));
    p.vecs = static_cast<int>(c.D / 8);
    p.W = with_labels ? reinterpret_cast<const uint4 *>(c.W) : nullptr;
    p.y = c.y + row0;
    p.V = c.V;
    p.ignore_index = c.ign;
    p.inv_t = c.inv_t;
    p.zx = c.zx;
    LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, c.s, launch_gather_rows(p, c.sms, c.s));
    return LCE_OK;
}

// Losses on answers have one chunk buffer. Where a cross-entropy call of that chunk would have two
// (no LCE_LOW_MEMORY) it holds twice the rows: the same memory, and what two chunks are split in for (the logits
// of one beside dH of the other) weighs less than contractions of twice the rows do where the rows that count are
// few: 1072 of 1531 rows x 50257 x 1600 under a frozen head 553 -> 375 us.
long long answer_chunk(long long N, long long chunk, int flags) {
    if (chunk <= 0 || N <= 0 || chunk >= N) return chunk;
    return (flags & LCE_LOW_MEMORY) ? chunk : chunk > N / 2 ? N : 2 * chunk;
}

// Losses on answers bring the rows that count together (prompts and padding are often half of a batch, and their
// rows cost as much as the others'): which rows they are, their labels, and a chunk's rows of H, at byte `at` of the
// workspace. Not done for so few rows that no tile of 256 would be saved, and
// not where chunks do not end on k blocks of the dW contraction.
struct GatherLayout {
    bool on = false;
    size_t off_rest = 0, off_next = 0, off_first = 0, off_index = 0, off_place = 0, off_labels = 0, off_H = 0, end = 0;
};

GatherLayout gather_layout(const Layout &L, long long N, long long D, long long V, bool gradient, size_t at) {
    GatherLayout g;
    g.on = N > 256 && (L.nchunks <= 1 || L.C % BK == 0);
    g.end = at;
    auto take = [&](size_t bytes) {
        const size_t o = g.end;
        g.end += align_up(bytes, 1024);
        return o;
    };
    if (gradient) {   // (of rows that are not brought together too)
        g.off_rest = take(sizeof(float) * static_cast<size_t>(L.C));
        g.off_next = take(sizeof(int) * static_cast<size_t>(L.C));
        g.off_first = take(sizeof(int) * static_cast<size_t>(L.frozen_w ? 0 : V));
    }
    if (!g.on) return g;
    g.off_index = take(sizeof(int) * static_cast<size_t>(N));
    g.off_place = take(sizeof(int) * static_cast<size_t>(N));
    g.off_labels = take(sizeof(long long) * static_cast<size_t>(N));
    g.off_H = take(2 * static_cast<size_t>(L.C) * static_cast<size_t>(D));
    return g;
}

void set_rests(Ctx &c, const GatherLayout &g, bool with_dw) {
    c.rests.rest = reinterpret_cast<float *>(c.ws + g.off_rest);
    c.rests.next = reinterpret_cast<int *>(c.ws + g.off_next);
    c.rests.first = with_dw ? reinterpret_cast<int *>(c.ws + g.off_first) : nullptr;
}

// H and y as setup gets them: the caller's, or their places in the workspace.
lce_status gather_inputs(const GatherLayout &g, const void *&H, const int64_t *&y, void *ws) {
    if (!g.on) return LCE_OK;
    if (!H || !y || !ws) return LCE_ERR_INVALID_ARG;
    if (!aligned16(H) || !aligned16(y)) return LCE_ERR_ALIGNMENT;
    H = static_cast<uint8_t *>(ws) + g.off_H;
    y = reinterpret_cast<const int64_t *>(static_cast<uint8_t *>(ws) + g.off_labels);
    return LCE_OK;
}

lce_status start_gather(Ctx &c, const GatherLayout &g, const void *H, const int64_t *y) {
    if (!g.on) return LCE_OK;
    c.Hrows = static_cast<const __nv_bfloat16 *>(H);
    c.index = reinterpret_cast<const int *>(c.ws + g.off_index);
    LCE_LAUNCH(launch_compact(reinterpret_cast<const long long *>(y), c.N, c.V, c.ign, c.hdr,
                              reinterpret_cast<int *>(c.ws + g.off_index), reinterpret_cast<int *>(c.ws + g.off_place),
                              reinterpret_cast<long long *>(c.ws + g.off_labels), c.s));
    return LCE_OK;
}

#define LCE_ZERO(ptr, bytes)                                                        \
    do {                                                                            \
        if (cudaMemsetAsync((ptr), 0, (bytes), c.s) != cudaSuccess) return LCE_ERR_CUDA; \
    } while (0)

// The gradients of chunks `first` (0 with two chunk buffers) .. n - 1 from a saved lse: each chunk's logits again, G straight
// from their epilogue, then the contractions. acc_dw0: dW is added to from the first one on.
lce_status backward_chunks(const Ctx &c, long long first, long long n, const float *lse, const float *dloss,
                           __nv_bfloat16 *dHb, bool acc_dh, float *dW, bool acc_dw0) {
    if (n <= first) return LCE_OK;
    if (frozen_overlapped(c)) {
        LCE_TRY(run_logits(c, MODE_G, 0, chunk_rows(c, 0), 0, lse, dloss, c.Gb[0]));
        for (long long k = 0; k < n; ++k) {
            const long long r0 = k * c.L.C, n0 = chunk_rows(c, k);
            GradSpec g{c.Gb[k & 1], c.Gb[k & 1], 0, true, true};
            LogitsSpec next{};
            if (k + 1 < n) {
                next = LogitsSpec{MODE_G, r0 + c.L.C, chunk_rows(c, k + 1),
                                  static_cast<int>(2 * k + 2), lse, dloss, c.Gb[(k + 1) & 1]};
                g.beside = &next;
            }
            LCE_TRY(run_grad(c, r0, n0, static_cast<int>(2 * k + 1), dHb + r0 * c.D, acc_dh, dW,
                             false, dloss, g));
        }
        return LCE_OK;
    }
    if (paired(c)) {
        // chunks in pairs (a, b): a's G (G epilogue) into buffer 0, its H^T into
        // columns 0..C-1; a's dH tiles, with b's logits (G into buffer 1) on the pairs
        // they leave free; b's H^T into columns C.., then b's dH beside one dW
        // contraction over both chunks (K = C + rows_b). An odd last chunk runs by itself.
        for (long long a = 0; a < n; a += 2) {
            const long long ra = a * c.L.C, na = chunk_rows(c, a);
            const bool has_b = a + 1 < n;
            const bool acc = a > 0 || acc_dw0;
            LCE_TRY(run_logits(c, MODE_G, ra, na, static_cast<int>(2 * a), lse, dloss, c.Gb[0]));
            LCE_TRY(run_transpose(c, ra, na, 0));
            if (!has_b) {
                LCE_TRY(run_grad(c, ra, na, static_cast<int>(2 * a + 1), dHb + ra * c.D, acc_dh, dW,
                                 acc, dloss, GradSpec{c.Gb[0], c.Gb[0], na, true, false}));
                break;
            }
            const long long b = a + 1, rb = b * c.L.C, nb = chunk_rows(c, b);
            // a's dH tiles, with b's logits tiles on the pairs they leave free
            const LogitsSpec lb{MODE_G, rb, nb, static_cast<int>(2 * b), lse, dloss, c.Gb[1]};
            GradSpec ga{c.Gb[0], c.Gb[0], 0, true, true};
            ga.beside = &lb;
            LCE_TRY(run_grad(c, ra, na, static_cast<int>(2 * a + 1), dHb + ra * c.D, acc_dh, dW,
                             acc, dloss, ga));
            LCE_TRY(run_transpose(c, rb, nb, c.L.C));
            LCE_TRY(run_grad(c, rb, nb, static_cast<int>(2 * b + 1), dHb + rb * c.D, acc_dh, dW,
                             acc, dloss, GradSpec{c.Gb[1], c.Gb[0], c.L.C + nb, true, false}));
        }
        return LCE_OK;
    }
    for (long long k = first; k < n; ++k) {
        const long long row0 = k * c.L.C;
        const long long rows = chunk_rows(c, k);
        LCE_TRY(bring_rows(c, k, false));
        LCE_TRY(run_logits(c, MODE_G, row0, rows, static_cast<int>(2 * k), lse, dloss, c.Gb[0]));
        LCE_TRY(run_grad(c, row0, rows, static_cast<int>(2 * k + 1), dHb + row0 * c.D, acc_dh, dW,
                         k > 0 || acc_dw0, dloss, GradSpec{c.Gb[0], c.Gb[0], rows, false, false}));
    }
    return LCE_OK;
}

}  // namespace

extern "C" {

lce_status lce_workspace_size(int64_t N, int64_t D, int64_t V, int64_t chunk, size_t *bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    Layout L;
    if (!make_layout(N, D, V, chunk, L)) return LCE_ERR_INVALID_ARG;
    *bytes = L.total;
    return LCE_OK;
}

lce_status lce_forward_workspace_size(int64_t N, int64_t D, int64_t V, int64_t chunk,
                                      size_t *bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    Layout L;
    if (!make_layout(N, D, V, chunk, L)) return LCE_ERR_INVALID_ARG;
    *bytes = L.fwd_total;
    return LCE_OK;
}

lce_status lce_count_valid(const int64_t *y, int64_t N, int64_t V, int64_t ignore_index,
                           int64_t *n_valid, lce_stream_t stream) {
    g_launches = 0;
    if (N < 0 || V <= 0 || !n_valid || (N > 0 && !y)) return LCE_ERR_INVALID_ARG;
    if ((y && !aligned16(y)) || (reinterpret_cast<uintptr_t>(n_valid) & 7u))
        return LCE_ERR_ALIGNMENT;
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s,
                    launch_count_valid(reinterpret_cast<const long long *>(y), N, V, ignore_index,
                                       reinterpret_cast<long long *>(n_valid), s));
    return LCE_OK;
}

lce_status lce_workspace_size_opt(int64_t N, int64_t D, int64_t V, int64_t chunk, int flags,
                                  size_t *bytes) {
    if (!bytes || (flags & ~LCE_FLAGS_ALL)) return LCE_ERR_INVALID_ARG;
    Layout L;
    if (!make_layout(N, D, V, chunk, L, (flags & LCE_FROZEN_W) != 0, (flags & LCE_LOW_MEMORY) != 0))
        return LCE_ERR_INVALID_ARG;
    *bytes = L.total + ((flags & LCE_ACCUMULATE_DH) ? acc_dh_bytes(L, D) : 0);
    return LCE_OK;
}

lce_status lce_forward_opt(const void *H, const void *W, const int64_t *y, int64_t N, int64_t D,
                           int64_t V, int64_t ignore_index, int64_t chunk, int reduction, int flags,
                           float *loss, float *lse, void *ws, size_t ws_bytes,
                           lce_stream_t stream) {
    g_launches = 0;
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    // nothing to accumulate here, and no chunk buffer to keep small
    if (flags & ~(LCE_INPUT_FP16 | LCE_LOW_MEMORY)) return LCE_ERR_INVALID_ARG;
    const bool none = reduction == LCE_REDUCTION_NONE;
    if ((!none && !loss) || (N > 0 && (!lse || !loss))) return LCE_ERR_INVALID_ARG;
    if ((loss && !aligned16(loss)) || (lse && !aligned16(lse))) return LCE_ERR_ALIGNMENT;
    Ctx c;
    LCE_TRY(setup(c, H, W, y, N, D, V, ignore_index, chunk, ws, ws_bytes, stream, false,
                  (flags & LCE_INPUT_FP16) != 0, false, true));
    c.reduction = reduction;
    float *rows_out = none ? loss : c.loss_rows;
    for (long long k = 0; k < c.L.nchunks; ++k) {
        const long long row0 = k * c.L.C;
        const long long rows = (c.N - row0) < c.L.C ? (c.N - row0) : c.L.C;
        LCE_TRY(run_logits(c, MODE_LSE, row0, rows, static_cast<int>(k), nullptr, nullptr,
                           c.Gb[0]));
        LCE_TRY(run_merge(c, row0, rows, lse, nullptr, rows_out));
    }
    if (!none)
        LCE_LAUNCH(launch_loss_finalize(c.loss_rows, c.N, c.hdr, loss,
                                        reduction == LCE_REDUCTION_MEAN, c.s));
    return LCE_OK;
}

lce_status lce_forward_ex(const void *H, const void *W, const int64_t *y, int64_t N, int64_t D,
                          int64_t V, int64_t ignore_index, int64_t chunk, int reduction,
                          float *loss, float *lse, void *ws, size_t ws_bytes,
                          lce_stream_t stream) {
    return lce_forward_opt(H, W, y, N, D, V, ignore_index, chunk, reduction, 0, loss, lse, ws,
                           ws_bytes, stream);
}

lce_status lce_forward(const void *H, const void *W, const int64_t *y, int64_t N, int64_t D,
                       int64_t V, int64_t ignore_index, int64_t chunk, float *loss, float *lse,
                       void *ws, size_t ws_bytes, lce_stream_t stream) {
    return lce_forward_ex(H, W, y, N, D, V, ignore_index, chunk, LCE_REDUCTION_MEAN, loss, lse, ws,
                          ws_bytes, stream);
}

lce_status lce_backward_opt(const void *H, const void *W, const int64_t *y, const float *lse,
                            const float *dloss, void *dH, float *dW, int64_t N, int64_t D,
                            int64_t V, int64_t ignore_index, int64_t chunk, int reduction,
                            int flags, void *ws, size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    if (flags & ~LCE_FLAGS_ALL) return LCE_ERR_INVALID_ARG;
    const bool f16 = (flags & LCE_INPUT_FP16) != 0;
    const bool frozen = (flags & LCE_FROZEN_W) != 0;
    if (frozen && (flags & LCE_ACCUMULATE_DW)) return LCE_ERR_INVALID_ARG;
    if (f16 && reduction == LCE_REDUCTION_NONE) return LCE_ERR_UNSUPPORTED;
    if ((!frozen && !dW) || (N > 0 && (!lse || !dH))) return LCE_ERR_INVALID_ARG;
    if ((dW && !aligned16(dW)) || (dH && !aligned16(dH)) || (lse && !aligned16(lse)))
        return LCE_ERR_ALIGNMENT;
    const bool low_mem = (flags & LCE_LOW_MEMORY) != 0;
    Layout L0;
    if (!make_layout(N, D, V, chunk, L0, frozen, low_mem)) return LCE_ERR_INVALID_ARG;
    if ((flags & LCE_ACCUMULATE_DH) && ws_bytes < L0.total + acc_dh_bytes(L0, D)) return LCE_ERR_WORKSPACE;
    Ctx c;
    LCE_TRY(setup(c, H, W, y, N, D, V, ignore_index, chunk, ws, ws_bytes, stream, false, f16,
                  frozen, false, low_mem));
    c.reduction = reduction;
    if (frozen) dW = nullptr;
    if (c.L.nchunks == 0 && dW && !(flags & LCE_ACCUMULATE_DW)) {
        if (cudaMemsetAsync(dW, 0, sizeof(float) * static_cast<size_t>(V) * D, c.s) != cudaSuccess)
            return LCE_ERR_CUDA;
    }
    return backward_chunks(c, 0, c.L.nchunks, lse, dloss, static_cast<__nv_bfloat16 *>(dH),
                           (flags & LCE_ACCUMULATE_DH) != 0, dW, (flags & LCE_ACCUMULATE_DW) != 0);
}

lce_status lce_backward_ex(const void *H, const void *W, const int64_t *y, const float *lse,
                           const float *dloss, void *dH, float *dW, int64_t N, int64_t D,
                           int64_t V, int64_t ignore_index, int64_t chunk, int reduction,
                           void *ws, size_t ws_bytes, lce_stream_t stream) {
    return lce_backward_opt(H, W, y, lse, dloss, dH, dW, N, D, V, ignore_index, chunk, reduction, 0,
                            ws, ws_bytes, stream);
}

lce_status lce_backward(const void *H, const void *W, const int64_t *y, const float *lse,
                        const float *dloss, void *dH, float *dW, int64_t N, int64_t D, int64_t V,
                        int64_t ignore_index, int64_t chunk, void *ws, size_t ws_bytes,
                        lce_stream_t stream) {
    return lce_backward_ex(H, W, y, lse, dloss, dH, dW, N, D, V, ignore_index, chunk,
                           LCE_REDUCTION_MEAN, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

// The fused call; n_valid_total (device int64, or null) replaces this call's own
// count of valid rows as the normaliser of the mean; pol: the policy loss in place of the
// cross-entropy (lse is then not written).
lce_status fwd_bwd_impl(const void *H, const void *W, const int64_t *y, const float *dloss,
                        int64_t N, int64_t D, int64_t V, int64_t ignore_index, int64_t chunk,
                        int reduction, int flags, float *loss, float *lse, void *dH, float *dW,
                        void *ws, size_t ws_bytes, lce_stream_t stream,
                        const int64_t *n_valid_total, const PolicyParams *pol = nullptr) {
    g_launches = 0;
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    if (flags & ~(LCE_FLAGS_ALL | (pol ? LCE_DW_BF16 : 0))) return LCE_ERR_INVALID_ARG;
    const bool f16 = (flags & LCE_INPUT_FP16) != 0;
    const bool frozen = (flags & LCE_FROZEN_W) != 0;
    const bool none = reduction == LCE_REDUCTION_NONE;
    if (frozen && (flags & LCE_ACCUMULATE_DW)) return LCE_ERR_INVALID_ARG;
    if (f16 && none) return LCE_ERR_UNSUPPORTED;
    if ((!none && !loss) || (!frozen && !dW) || (N > 0 && ((!lse && !pol) || !dH || !loss)))
        return LCE_ERR_INVALID_ARG;
    if ((loss && !aligned16(loss)) || (dW && !aligned16(dW)) || (dH && !aligned16(dH)) ||
        (lse && !aligned16(lse)))
        return LCE_ERR_ALIGNMENT;
    const bool acc_dh = (flags & LCE_ACCUMULATE_DH) != 0;
    const bool low_mem = pol || (flags & LCE_LOW_MEMORY) != 0;
    if (pol) chunk = answer_chunk(N, chunk, flags);
    Layout L0;
    if (!make_layout(N, D, V, chunk, L0, frozen, low_mem, pol != nullptr)) return LCE_ERR_INVALID_ARG;
    if (acc_dh && ws_bytes < L0.total + acc_dh_bytes(L0, D)) return LCE_ERR_WORKSPACE;
    GatherLayout gl;
    const void *Hs = H;
    const int64_t *ys = y;
    if (pol) {
        gl = gather_layout(L0, N, D, V, true, L0.total + acc_dh_bytes(L0, D));
        if (ws_bytes < gl.end) return LCE_ERR_WORKSPACE;
        if ((flags & LCE_DW_BF16) && (frozen || (flags & LCE_ACCUMULATE_DW) || L0.nchunks > 1)) return LCE_ERR_UNSUPPORTED;
        LCE_TRY(gather_inputs(gl, Hs, ys, ws));
    }
    Ctx c;
    LCE_TRY(setup(c, Hs, W, ys, N, D, V, ignore_index, chunk, ws, ws_bytes, stream, gl.on, f16,
                  frozen, false, low_mem, !gl.on, pol != nullptr));
    c.reduction = reduction;
    if (pol) {
        c.pol = *pol;
        c.inv_t = pol->inv_t;
        c.answers = true;
        set_rests(c, gl, !frozen);
        c.dw16 = (flags & LCE_DW_BF16) != 0;
        LCE_TRY(start_gather(c, gl, H, y));
        if (gl.on) {   // what rows that do not count have
            c.loss_by_index = none;
            LCE_ZERO(none ? loss : c.loss_rows, sizeof(float) * static_cast<size_t>(N));
            LCE_ZERO(pol->logp, sizeof(float) * static_cast<size_t>(N));
            if (!acc_dh) LCE_ZERO(dH, 2 * static_cast<size_t>(N) * static_cast<size_t>(D));
        }
    }
    if (n_valid_total) LCE_LAUNCH(launch_set_nvalid(reinterpret_cast<const long long *>(n_valid_total),
                                                    c.hdr, c.s));
    if (frozen) dW = nullptr;
    float *rows_out = none ? loss : c.loss_rows;
    if (c.L.nchunks == 0 && dW && !(flags & LCE_ACCUMULATE_DW)) {
        if (cudaMemsetAsync(dW, 0, (c.dw16 ? 2 : sizeof(float)) * static_cast<size_t>(V) * D, c.s) != cudaSuccess)
            return LCE_ERR_CUDA;
    }
    const bool acc_dw0 = (flags & LCE_ACCUMULATE_DW) != 0;
    __nv_bfloat16 *dHb = static_cast<__nv_bfloat16 *>(dH);
    if (frozen_overlapped(c)) {
        // chunk k's dH tiles, with chunk k+1's logits (P' into buffer (k+1) % 2) on
        // the pairs they leave free; then chunk k+1's prep (no H^T: no dW)
        LCE_TRY(run_logits(c, MODE_LSE_P, 0, chunk_rows(c, 0), 0, nullptr, nullptr, c.Gb[0]));
        LCE_TRY(run_prep(c, 0, chunk_rows(c, 0), lse, dloss, rows_out, c.Gb[0], false));
        for (long long k = 0; k < c.L.nchunks; ++k) {
            const long long r0 = k * c.L.C, n0 = chunk_rows(c, k);
            GradSpec g{c.Gb[k & 1], c.Gb[k & 1], 0, true, true};
            LogitsSpec next{};
            if (k + 1 < c.L.nchunks) {
                next = LogitsSpec{MODE_LSE_P, r0 + c.L.C, chunk_rows(c, k + 1),
                                  static_cast<int>(2 * k + 2), nullptr, nullptr, c.Gb[(k + 1) & 1]};
                g.beside = &next;
            }
            LCE_TRY(run_grad(c, r0, n0, static_cast<int>(2 * k + 1), dHb + r0 * c.D, acc_dh, dW,
                             false, dloss, g));
            if (k + 1 < c.L.nchunks)
                LCE_TRY(run_prep(c, r0 + c.L.C, chunk_rows(c, k + 1), lse, dloss, rows_out,
                                 c.Gb[(k + 1) & 1], false));
        }
    } else if (paired(c)) {
        // chunks in pairs (a, b): a's P' into buffer 0, its prep (lse, row losses,
        // P' -> G, H^T into columns 0..C-1); a's dH tiles, with b's logits (P' into
        // buffer 1) on the pairs they leave free; b's prep (H^T into columns C..), then
        // b's dH beside one dW contraction over both chunks (K = C + rows_b). An odd
        // last chunk runs by itself.
        for (long long a = 0; a < c.L.nchunks; a += 2) {
            const long long ra = a * c.L.C, na = chunk_rows(c, a);
            const bool has_b = a + 1 < c.L.nchunks;
            const bool acc = a > 0 || acc_dw0;
            LCE_TRY(run_logits(c, MODE_LSE_P, ra, na, static_cast<int>(2 * a), nullptr, nullptr,
                               c.Gb[0]));
            LCE_TRY(run_prep(c, ra, na, lse, dloss, rows_out, c.Gb[0], true, 0));
            if (!has_b) {
                LCE_TRY(run_grad(c, ra, na, static_cast<int>(2 * a + 1), dHb + ra * c.D, acc_dh, dW,
                                 acc, dloss, GradSpec{c.Gb[0], c.Gb[0], na, true, false}));
                break;
            }
            const long long b = a + 1, rb = b * c.L.C, nb = chunk_rows(c, b);
            // a's dH tiles, with b's logits tiles on the pairs they leave free
            const LogitsSpec lb{MODE_LSE_P, rb, nb, static_cast<int>(2 * b), nullptr, nullptr,
                                c.Gb[1]};
            GradSpec ga{c.Gb[0], c.Gb[0], 0, true, true};
            ga.beside = &lb;
            LCE_TRY(run_grad(c, ra, na, static_cast<int>(2 * a + 1), dHb + ra * c.D, acc_dh, dW,
                             acc, dloss, ga));
            LCE_TRY(run_prep(c, rb, nb, lse, dloss, rows_out, c.Gb[1], true, c.L.C));
            LCE_TRY(run_grad(c, rb, nb, static_cast<int>(2 * b + 1), dHb + rb * c.D, acc_dh, dW,
                             acc, dloss, GradSpec{c.Gb[1], c.Gb[0], c.L.C + nb, true, false}));
        }
    } else {
        for (long long k = 0; k < c.L.nchunks; ++k) {
            const long long row0 = k * c.L.C;
            const long long rows = chunk_rows(c, k);
            LCE_TRY(bring_rows(c, k, false));
            LCE_TRY(run_logits(c, MODE_LSE_P, row0, rows, static_cast<int>(2 * k), nullptr, nullptr,
                               c.Gb[0]));
            LCE_TRY(run_prep(c, row0, rows, lse, dloss, rows_out, c.Gb[0], !frozen));
            LCE_TRY(run_grad(c, row0, rows, static_cast<int>(2 * k + 1), dHb + row0 * c.D, acc_dh,
                             dW, k > 0 || acc_dw0, dloss,
                             GradSpec{c.Gb[0], c.Gb[0], frozen ? 0 : rows, true, false}));
        }
    }
    if (!none)
        LCE_LAUNCH(launch_loss_finalize(c.loss_rows, c.N, c.hdr, loss,
                                        reduction == LCE_REDUCTION_MEAN, c.s));
    return LCE_OK;
}

// (the largest logit over the temperature has to stay within fp32: logits up to 1.2e19)
constexpr float POLICY_MIN_TEMPERATURE = 0x1p-64f;

// Checks of the policy's vectors and numbers (advantages may be null with no rows).
lce_status policy_check(int64_t N, const float *advantages, const float *old_logprobs, const float *ref_logprobs,
                        const float *weights, float clip_low, float clip_high, float beta, float temperature,
                        const float *logprobs) {
    if (N > 0 && (!advantages || !logprobs)) return LCE_ERR_INVALID_ARG;
    if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f && clip_high < INFINITY) ||
        !(beta >= 0.f && beta < INFINITY) || !(temperature >= POLICY_MIN_TEMPERATURE && temperature < INFINITY))
        return LCE_ERR_INVALID_ARG;
    if (N > 0 && beta != 0.f && !ref_logprobs) return LCE_ERR_INVALID_ARG;
    const uintptr_t words = reinterpret_cast<uintptr_t>(advantages) | reinterpret_cast<uintptr_t>(old_logprobs) |
                            reinterpret_cast<uintptr_t>(ref_logprobs) | reinterpret_cast<uintptr_t>(weights) |
                            reinterpret_cast<uintptr_t>(logprobs);
    return words % 4 ? LCE_ERR_ALIGNMENT : LCE_OK;
}

PolicyParams policy_params(const float *advantages, const float *old_logprobs, const float *ref_logprobs,
                           const float *weights, float clip_low, float clip_high, float beta, float temperature,
                           float *logprobs) {
    PolicyParams p;
    p.adv = advantages;
    p.old_logp = old_logprobs;
    p.ref_logp = beta != 0.f ? ref_logprobs : nullptr;
    p.weight = weights;
    p.lo = 1.f - clip_low;
    p.hi = 1.f + clip_high;
    p.beta = beta;
    p.inv_t = 1.f / temperature;
    p.logp = logprobs;
    return p;
}

// Workspace of a preference over the head: the loss path's layout (the forward's share of it
// without gradients), then lse and the coefficient of each row, and the pairs' losses.
struct PrefLayout {
    Layout L;
    GatherLayout gather;
    size_t off_lse = 0, off_zx = 0, off_fix = 0, off_coef = 0, off_pair = 0, off_clean = 0, total = 0;
};

// (chunk: as answer_chunk has it)
bool make_pref_layout(int64_t N, int64_t D, int64_t V, int64_t chunk, int64_t pairs, int flags, bool grad,
                      PrefLayout &P) {
    if (!make_layout(N, D, V, chunk, P.L, (flags & LCE_FROZEN_W) != 0, true, true) || pairs <= 0 || pairs > (1ll << 24)) return false;
    const size_t rows = sizeof(float) * static_cast<size_t>(N > 0 ? N : 1);
    P.gather = gather_layout(P.L, N, D, V, grad, grad ? P.L.total + acc_dh_bytes(P.L, D) : P.L.fwd_total);
    size_t off = P.gather.end;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align_up(bytes, 1024);
        return at;
    };
    P.off_lse = take(rows);
    P.off_zx = take(sizeof(float) * static_cast<size_t>(P.L.C > 0 ? P.L.C : 1));
    P.off_fix = take(2 * rows);
    P.off_pair = take(sizeof(float) * static_cast<size_t>(pairs));
    P.off_clean = take(sizeof(int) * static_cast<size_t>(2 * pairs + 1));
    if (grad) P.off_coef = take(rows);
    P.total = off;
    return true;
}

lce_status preference_check(const int64_t *offsets, int64_t pairs, const float *ref_logprobs, float beta,
                            float label_smoothing, int reduction, const float *dloss, const float *loss,
                            const float *seq_logprobs) {
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    if (pairs <= 0 || !offsets || !loss || !seq_logprobs) return LCE_ERR_INVALID_ARG;
    if (!(beta > -INFINITY && beta < INFINITY) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
        return LCE_ERR_INVALID_ARG;
    const uintptr_t words = reinterpret_cast<uintptr_t>(ref_logprobs) | reinterpret_cast<uintptr_t>(dloss) |
                            reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(seq_logprobs);
    return words % 4 || reinterpret_cast<uintptr_t>(offsets) % 8 ? LCE_ERR_ALIGNMENT : LCE_OK;
}

PairParams pair_params(const int64_t *offsets, int64_t pairs, int64_t N, int64_t V, int64_t ign, const int64_t *y,
                       const float *loss_rows, const float *ref, float beta, float smoothing, int average,
                       const float *dloss, int reduction, float *loss, float *seq, float *pair_loss, int *clean,
                       float *coef, int *hdr) {
    const bool none = reduction == LCE_REDUCTION_NONE;
    PairParams p;
    p.offsets = reinterpret_cast<const long long *>(offsets);
    p.clean = pairs > PAIRS_BY_THEMSELVES ? clean : nullptr;
    p.pairs = pairs;
    p.N = N;
    p.V = V;
    p.ignore_index = ign;
    p.y = reinterpret_cast<const long long *>(y);
    p.loss_rows = loss_rows;
    p.place = nullptr;
    p.fix = nullptr;
    p.ref = ref;
    p.beta = beta;
    p.smoothing = smoothing;
    p.average = average ? 1 : 0;
    p.dloss = dloss;
    p.dloss_per_pair = none ? 1 : 0;
    p.mean = reduction == LCE_REDUCTION_MEAN ? 1 : 0;
    p.seq_logp = seq;
    p.pair_loss = none ? loss : pair_loss;
    p.loss = none ? nullptr : loss;
    p.coef = coef;
    p.hdr = hdr;
    return p;
}

// ---- 8-bit product
lce_status fp8_matmul_check(const void *A, int64_t lda, const float *sa, int64_t sa_row, int64_t sa_block,
                            const void *B, int64_t ldb, const float *sb, int64_t sb_row, int64_t sb_block,
                            int64_t M, int64_t N, int64_t K, const void *out, int64_t ldc, int c_dtype,
                            const void *ws, size_t ws_bytes) {
    if (sa_row < 0 || sa_block < 0 || sb_row < 0 || sb_block < 0) return LCE_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K <= 0 || M > MAX_V || N > MAX_V || K > MAX_V) return LCE_ERR_INVALID_ARG;
    if (lda < K || ldb < K || ldc < N || c_dtype < CE_BF16 || c_dtype > CE_FP16 || !ws)
        return LCE_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (!A || !sa || !B || !sb || !out)) return LCE_ERR_INVALID_ARG;
    const int64_t elem = c_dtype == CE_FP32 ? 4 : 2;
    if (!aligned16(A) || !aligned16(B) || !aligned16(out) || !aligned16(ws) || lda % 16 || ldb % 16 ||
        (ldc * elem) % 16 || reinterpret_cast<uintptr_t>(sa) % 4 || reinterpret_cast<uintptr_t>(sb) % 4)
        return LCE_ERR_ALIGNMENT;
    if (ws_bytes < 1024) return LCE_ERR_WORKSPACE;
    return LCE_OK;
}

// In how many parts of k the tiles of a product by CTA pairs are taken (tile scales only): what the
// last, partly filled wave of tiles leaves idle is shared out. One wave of tiles takes 0.46 us per
// k block, the parts are written and read at about 5 bytes per ns, and their sum is one
// launch. (us, one part / as chosen: 1531 x 1600 x 50257, 42 tiles for 76 pairs, 182 / 145; 700 x 4001 x 33001
// 124 / 102; 1537 x 1701 x 20000 79 / 69; 2049 x 1290 x 50000 184 / 165.)
int fp8_parts(long long tiles, long long M, long long N, long long KB, int pairs) {
    int best = 1;
    double best_us = 1e30;
    for (int n = 1; n <= 8 && KB >= 16 * n; ++n) {
        const double us = 0.46 * static_cast<double>(cdiv(tiles * n, pairs)) * static_cast<double>(cdiv(KB, n)) +
                          (n > 1 ? 5.0 + 8.0 * n * static_cast<double>(M) * static_cast<double>(N) / 5e6 : 0.0);
        if (us < best_us * 0.97) {
            best = n;
            best_us = us;
        }
    }
    return best;
}
bool fp8_pairs(int64_t M, int64_t N, int sms, int pairs) {
    // Pairs of CTAs as soon as 128 x 128 tiles would not all run at once (us, tiles / pairs: 512 x 4864 x 4096,
    // 152 tiles, 18.5 / 20.2; 1531 x 1600 x 4096, 156 tiles, 29.0 / 20.2; 200 x 32000 x 4096 52 / 40;
    // 256 x 4864 x 4096 14.9 / 19.7). Up to 128 rows half of a pair would have none.
    return M > 128 && pairs > 0 && cdiv(M, 128) * cdiv(N, 128) > sms;
}
size_t fp8_parts_bytes(int64_t M, int64_t N, int parts) {
    return parts > 1 ? sizeof(float) * static_cast<size_t>(parts) * cdiv(M, 256) * 256 *
                           align_up(static_cast<size_t>(N), 32) : 0;
}

// ws: the header and what follows it; parts: where the sums of a product in parts may lie (fp32, 16-byte
// aligned; nothing else of this call), parts_bytes long
// after_quantize: A comes from the quantisation launched just before on the same stream,
// which the product's prologue may overlap
lce_status fp8_matmul(const void *A, int64_t lda, const float *sa, int64_t sa_row, int64_t sa_block,
                      const void *B, int64_t ldb, const float *sb, int64_t sb_row, int64_t sb_block,
                      int b_rows, int64_t M, int64_t N, int64_t K, void *out, int64_t ldc, int c_dtype,
                      void *ws, size_t ws_bytes, void *parts, size_t parts_bytes, bool after_quantize,
                      lce_stream_t stream) {
    lce_status st = fp8_matmul_check(A, lda, sa, sa_row, sa_block, B, ldb, sb, sb_row, sb_block, M, N, K, out, ldc,
                                     c_dtype, ws, ws_bytes);
    if (st != LCE_OK) return st;
    const int64_t elem = c_dtype == CE_FP32 ? 4 : 2;
    int sms = 0, pairs = 0;
    st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    if (!fp8_ready()) return LCE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0 || N == 0)
        return cudaMemsetAsync(ws, 0, sizeof(int), s) == cudaSuccess ? LCE_OK : LCE_ERR_CUDA;

    Fp8GemmParams p;
    memset(&p, 0, sizeof(p));
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.KB = static_cast<int>(cdiv(K, 128));
    const long long pair_tiles = cdiv(M, 256) * cdiv(N, 256), tiles = cdiv(M, 128) * cdiv(N, 128);
    const bool pair = fp8_pairs(M, N, sms, pairs);
    if (tiles > 0x7fffffffll) return LCE_ERR_INVALID_ARG;
    // A tile is split along k over 2, 4 or 8 CTAs while all run at once and each keeps 2 k blocks (us,
    // split in 1 / 2 / 4 / 8: 8 x 1600 x 50257, 13 tiles, 126 / 67 / 37 / 23; 64 x 4096 x 4096, 32 tiles, 16.9 /
    // 13.4 / 9.7 / 22.7; 64 x 12800 x 4096, 100 tiles, 18.6 / 29.2 / 29.5 / 54).
    int split = 1;
    if (!pair)
        while (split < 8 && tiles * split * 2 <= sms && p.KB >= split * 4) split *= 2;
    p.m_tiles = static_cast<int>(pair ? cdiv(M, 256) : cdiv(M, 128));
    p.n_tiles = static_cast<int>(pair ? cdiv(N, 256) : cdiv(N, 128));
    p.tiles = static_cast<int>(pair ? pair_tiles : tiles);
    p.a_box_rows = pair || M >= 128 ? 128 : static_cast<int>(align_up(static_cast<size_t>(M), 8));
    p.n_bulk = static_cast<int>(N / (16 / elem) * (16 / elem));
    // what 192 KB hold of A's rows and 128 rows of B (a multiple of 1 KB each), as barriers allow (6 stages /
    // 11: 1 x 128256 x 4096 86.7 / 83.7 us, 64 x 128256 x 4096 96.3 / 94.9, 1 x 32000 x 4096 27.6 / 28.0)
    p.stages = std::min(11, 6 * 32768 / (p.a_box_rows * 128 + 16384));
    p.sa = sa;
    p.sb = sb;
    p.sa_row = sa_row;
    p.sa_block = sa_block;
    p.sb_row = sb_row;
    p.sb_block = sb_block;
    // (as quantize_fp8 stores them: 4096 x 8192 x 4096 183 us, one by one 241)
    p.sb_vec = sb_row == 1 && sb_block % 4 == 0 && aligned16(sb) ? 1 : 0;
    p.C = out;
    p.ldc = ldc;
    p.c_type = c_dtype;
    p.hdr = static_cast<int *>(ws);
    p.timeout_ns = kDefaultTimeoutNs;
    p.parts = pair && !b_rows ? fp8_parts(pair_tiles, M, N, p.KB, pairs) : 1;
    if (p.parts > 1 && parts_bytes < fp8_parts_bytes(M, N, p.parts)) p.parts = 1;
    if (p.parts > 1) {
        p.C = parts;
        p.ldc = static_cast<long long>(align_up(static_cast<size_t>(N), 32));
        p.c_type = CE_FP32;
        p.n_bulk = static_cast<int>(p.ldc);
    }
    const MapType ct = p.c_type == CE_FP32 ? MAP_F32 : c_dtype == CE_FP16 ? MAP_F16 : MAP_BF16;
    const long long c_rows = p.parts > 1 ? static_cast<long long>(p.parts) * p.m_tiles * 256 : M;
    if (!encode_2d(&p.tmA, A, K, M, lda, 128, p.a_box_rows, MAP_U8) ||
        !encode_2d(&p.tmB, B, K, N, ldb, 128, 128, MAP_U8) ||
        (p.n_bulk > 0 &&
         !encode_store_2d(&p.tmC, p.C, p.n_bulk, c_rows, p.ldc * (p.c_type == CE_FP32 ? 4 : 2), ct, 32)))
        return LCE_ERR_CUDA;
    const int cluster = pair ? 2 : split;
    const int most = pair ? pairs : split > 1 ? p.tiles : sms;
    const long long units = static_cast<long long>(p.tiles) * p.parts;
    const int clusters = static_cast<int>(units < most ? units : most);
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_fp8_matmul(p, pair, b_rows != 0, cluster, clusters, after_quantize, s));
    if (p.parts > 1) LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_fp8_parts(p, out, ldc, c_dtype, s));
    return LCE_OK;
}

// ---- gradient norm and clipping
constexpr int64_t kMaxGrads = 1 << 20;

// Whether a written tensor overlaps another tensor of the call (an output may be its
// own gradient).
struct Range {
    uintptr_t a, b;   // bytes [a, b)
    bool written;
};
lce_status check_overlap(const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                         void *const *outs, int64_t n) {
    std::unique_ptr<Range[]> r(new (std::nothrow) Range[static_cast<size_t>(2 * n)]);
    if (!r) return LCE_ERR_CUDA;
    int64_t k = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (!sizes[i]) continue;
        const uintptr_t bytes = static_cast<uintptr_t>(sizes[i]) * (dtypes[i] == CE_FP32 ? 4 : 2);
        const uintptr_t in = reinterpret_cast<uintptr_t>(grads[i]);
        const uintptr_t out = outs ? reinterpret_cast<uintptr_t>(outs[i]) : in;
        r[k++] = {out, out + bytes, true};
        if (out != in) r[k++] = {in, in + bytes, false};
    }
    std::sort(r.get(), r.get() + k, [](const Range &x, const Range &y) { return x.a < y.a; });
    uintptr_t end = 0, written_end = 0;   // of the ranges so far
    for (int64_t i = 0; i < k; ++i) {
        if (r[i].a < (r[i].written ? end : written_end)) return LCE_ERR_INVALID_ARG;
        end = std::max(end, r[i].b);
        if (r[i].written) written_end = std::max(written_end, r[i].b);
    }
    return LCE_OK;
}

lce_status grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                     void *const *outs, int64_t n, int kind, bool clip, float max_norm, float eps,
                     float *norm, void *ws, size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    if (n < 0 || n > kMaxGrads || !norm || !ws) return LCE_ERR_INVALID_ARG;
    if (n > 0 && (!grads || !sizes || !dtypes)) return LCE_ERR_INVALID_ARG;
    if (kind < LCE_NORM_2 || kind > LCE_NORM_1) return LCE_ERR_INVALID_ARG;
    bool copy = false;
    for (int64_t i = 0; i < n; ++i) {
        if (dtypes[i] < CE_BF16 || dtypes[i] > CE_FP16) return LCE_ERR_INVALID_ARG;
        if (sizes[i] < 0 || sizes[i] > (1ll << 40)) return LCE_ERR_INVALID_ARG;
        if (!sizes[i]) continue;
        if (!grads[i] || (outs && !outs[i])) return LCE_ERR_INVALID_ARG;
        const uintptr_t elem = dtypes[i] == CE_FP32 ? 4 : 2;
        if (reinterpret_cast<uintptr_t>(grads[i]) % elem) return LCE_ERR_ALIGNMENT;
        if (outs && reinterpret_cast<uintptr_t>(outs[i]) % elem) return LCE_ERR_ALIGNMENT;
        copy |= outs && outs[i] != grads[i];
    }
    if (!aligned16(ws) || reinterpret_cast<uintptr_t>(norm) % 4) return LCE_ERR_ALIGNMENT;
    if (ws_bytes < static_cast<size_t>(n > 0 ? cdiv(n, CLIP_MAX_TENSORS) : 1) * CLIP_MAX_PARTS * sizeof(double))
        return LCE_ERR_WORKSPACE;
    if (clip) {
        const lce_status ov = check_overlap(grads, sizes, dtypes, outs, n);
        if (ov != LCE_OK) return ov;
    }
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    double *part = static_cast<double *>(ws);
    ClipItem items[CLIP_MAX_TENSORS];
    // the next tensors of one launch, from tensor i on; returns the tensor after them
    auto batch = [&](int64_t i, int *m) {
        *m = 0;
        long long chunks = 0;
        for (; i < n && *m < CLIP_MAX_TENSORS; ++i) {
            if (!sizes[i]) continue;
            const long long c = clip_chunks(grads[i], sizes[i], dtypes[i]);
            if (*m > 0 && chunks + c > CLIP_MAX_CHUNKS) break;
            chunks += c;
            items[(*m)++] = {grads[i], outs ? outs[i] : const_cast<void *>(grads[i]), sizes[i], dtypes[i], c};
        }
        return i;
    };
    int nparts = 0, m = 0;
    int64_t i = 0;
    bool one_batch = true;
    do {
        i = batch(i, &m);
        one_batch = one_batch && i >= n;
        if (nparts + CLIP_MAX_PARTS > static_cast<long long>(ws_bytes / sizeof(double))) return LCE_ERR_WORKSPACE;
        if (m > 0) {
            int wrote = 0;
            LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s,
                            launch_grad_norm(items, m, kind, part + nparts, sms, &wrote, s));
            nparts += wrote;
        }
    } while (i < n);
    ClipScale c;
    c.kind = kind;
    c.part = part;
    c.nparts = nparts;
    c.max_norm = max_norm;
    c.eps = eps;
    c.copy = copy ? 1 : 0;
    c.tell = 1;
    c.norm_out = norm;
    if (!clip) {
        LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_grad_scale(items, 0, c, sms, s));
        return LCE_OK;
    }
    i = 0;
    do {
        if (!one_batch) i = batch(i, &m);
        else i = n;
        LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_grad_scale(items, m, c, sms, s));
        c.tell = 0;
    } while (i < n);
    return LCE_OK;
}

}  // namespace

extern "C" {

lce_status lce_fwd_bwd_opt(const void *H, const void *W, const int64_t *y, const float *dloss,
                           int64_t N, int64_t D, int64_t V, int64_t ignore_index, int64_t chunk,
                           int reduction, int flags, float *loss, float *lse, void *dH, float *dW,
                           void *ws, size_t ws_bytes, lce_stream_t stream) {
    return fwd_bwd_impl(H, W, y, dloss, N, D, V, ignore_index, chunk, reduction, flags, loss, lse,
                        dH, dW, ws, ws_bytes, stream, nullptr);
}

lce_status lce_fwd_bwd_sharded(const void *H, const void *W, const int64_t *y, const float *dloss,
                               const int64_t *n_valid_total, int64_t N, int64_t D, int64_t V,
                               int64_t ignore_index, int64_t chunk, int flags, float *loss,
                               float *lse, void *dH, float *dW, void *ws, size_t ws_bytes,
                               lce_stream_t stream) {
    g_launches = 0;
    if (!n_valid_total) return LCE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(n_valid_total) & 7u) return LCE_ERR_ALIGNMENT;
    return fwd_bwd_impl(H, W, y, dloss, N, D, V, ignore_index, chunk, LCE_REDUCTION_MEAN, flags,
                        loss, lse, dH, dW, ws, ws_bytes, stream, n_valid_total);
}

lce_status lce_fwd_bwd_ex(const void *H, const void *W, const int64_t *y, const float *dloss,
                          int64_t N, int64_t D, int64_t V, int64_t ignore_index, int64_t chunk,
                          int reduction, float *loss, float *lse, void *dH, float *dW, void *ws,
                          size_t ws_bytes, lce_stream_t stream) {
    return lce_fwd_bwd_opt(H, W, y, dloss, N, D, V, ignore_index, chunk, reduction, 0, loss, lse,
                           dH, dW, ws, ws_bytes, stream);
}

lce_status lce_fwd_bwd(const void *H, const void *W, const int64_t *y, const float *dloss,
                       int64_t N, int64_t D, int64_t V, int64_t ignore_index, int64_t chunk,
                       float *loss, float *lse, void *dH, float *dW, void *ws, size_t ws_bytes,
                       lce_stream_t stream) {
    return lce_fwd_bwd_ex(H, W, y, dloss, N, D, V, ignore_index, chunk, LCE_REDUCTION_MEAN, loss,
                          lse, dH, dW, ws, ws_bytes, stream);
}

lce_status lce_policy_workspace_size(int64_t N, int64_t D, int64_t V, int64_t chunk, int flags, int gradient,
                                     size_t *bytes) {
    Layout L;
    if (!bytes || (flags & ~(LCE_FLAGS_ALL | LCE_DW_BF16)) ||
        !make_layout(N, D, V, gradient ? answer_chunk(N, chunk, flags) : chunk, L, (flags & LCE_FROZEN_W) != 0, true, true))
        return LCE_ERR_INVALID_ARG;
    *bytes = gather_layout(L, N, D, V, gradient != 0, gradient ? L.total + acc_dh_bytes(L, D) : L.fwd_total).end;
    return LCE_OK;
}

lce_status lce_policy_forward(const void *H, const void *W, const int64_t *y, const float *advantages,
                              const float *old_logprobs, const float *ref_logprobs, const float *weights,
                              float clip_low, float clip_high, float beta, float temperature, int64_t N,
                              int64_t D, int64_t V, int64_t ignore_index, int64_t chunk, int reduction,
                              float *loss, float *logprobs, void *ws, size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    const bool none = reduction == LCE_REDUCTION_NONE;
    if (!loss && (N > 0 || !none)) return LCE_ERR_INVALID_ARG;
    if (loss && !aligned16(loss)) return LCE_ERR_ALIGNMENT;
    LCE_TRY(policy_check(N, advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta,
                         temperature, logprobs));
    Layout L0;
    if (!make_layout(N, D, V, chunk, L0, false, true)) return LCE_ERR_INVALID_ARG;
    const GatherLayout gl = gather_layout(L0, N, D, V, false, L0.fwd_total);
    if (ws_bytes < gl.end) return LCE_ERR_WORKSPACE;
    const void *Hs = H;
    const int64_t *ys = y;
    LCE_TRY(gather_inputs(gl, Hs, ys, ws));
    Ctx c;
    LCE_TRY(setup(c, Hs, W, ys, N, D, V, ignore_index, chunk, ws, ws_bytes, stream, gl.on, false, false, true, true,
                  !gl.on));
    c.reduction = reduction;
    LCE_TRY(start_gather(c, gl, H, y));
    if (gl.on) {   // what rows that do not count have
        c.loss_by_index = none;
        LCE_ZERO(none ? loss : c.loss_rows, sizeof(float) * static_cast<size_t>(N));
        LCE_ZERO(logprobs, sizeof(float) * static_cast<size_t>(N));
    }
    c.pol = policy_params(advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta,
                          temperature, logprobs);
    c.inv_t = c.pol.inv_t;
    c.answers = true;
    for (long long k = 0; k < c.L.nchunks; ++k) {
        LCE_TRY(bring_rows(c, k, false));
        LCE_TRY(run_logits(c, MODE_LSE, k * c.L.C, chunk_rows(c, k), static_cast<int>(k), nullptr, nullptr,
                           c.Gb[0]));
        LCE_TRY(run_merge(c, k * c.L.C, chunk_rows(c, k), nullptr, nullptr, none ? loss : c.loss_rows));
    }
    if (!none)
        LCE_LAUNCH(launch_loss_finalize(c.loss_rows, c.N, c.hdr, loss, reduction == LCE_REDUCTION_MEAN, c.s));
    return LCE_OK;
}

lce_status lce_policy_fwd_bwd(const void *H, const void *W, const int64_t *y, const float *advantages,
                              const float *old_logprobs, const float *ref_logprobs, const float *weights,
                              float clip_low, float clip_high, float beta, float temperature,
                              const float *dloss, int64_t N, int64_t D, int64_t V, int64_t ignore_index,
                              int64_t chunk, int reduction, int flags, float *loss, float *logprobs, void *dH,
                              void *dW, void *ws, size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    // (16-bit floats: a policy's coefficients have no range that fp16 gradients could be scaled by)
    if (flags & LCE_INPUT_FP16) return LCE_ERR_UNSUPPORTED;
    LCE_TRY(policy_check(N, advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta,
                         temperature, logprobs));
    const PolicyParams pol = policy_params(advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high,
                                           beta, temperature, logprobs);
    return fwd_bwd_impl(H, W, y, dloss, N, D, V, ignore_index, chunk, reduction, flags, loss, nullptr, dH,
                        static_cast<float *>(dW), ws, ws_bytes, stream, nullptr, &pol);
}

lce_status lce_preference_workspace_size(int64_t N, int64_t D, int64_t V, int64_t chunk, int64_t pairs, int flags,
                                         int gradient, size_t *bytes) {
    PrefLayout P;
    if (!bytes || (flags & ~(LCE_FLAGS_ALL | LCE_DW_BF16)) ||
        !make_pref_layout(N, D, V, gradient ? answer_chunk(N, chunk, flags) : chunk, pairs, flags, gradient != 0, P))
        return LCE_ERR_INVALID_ARG;
    *bytes = P.total;
    return LCE_OK;
}

// Phases: every chunk's logits and the rows' log probabilities; the pairs; the gradients. The first chunk comes last in
// the first phase and stays in the chunk buffer over the pairs, so that its logits are not computed
// again: with no more rows than the buffer holds, none are.
lce_status lce_preference_fwd_bwd(const void *H, const void *W, const int64_t *y, const int64_t *offsets,
                                  int64_t pairs, const float *ref_logprobs, float beta, float label_smoothing,
                                  int average, const float *dloss, int64_t N, int64_t D, int64_t V,
                                  int64_t ignore_index, int64_t chunk, int reduction, int flags, float *loss,
                                  float *seq_logprobs, void *dH, void *dW_, void *ws, size_t ws_bytes,
                                  lce_stream_t stream) {
    g_launches = 0;
    float *dW = static_cast<float *>(dW_);   // (bf16 with LCE_DW_BF16)
    if (flags & ~(LCE_FLAGS_ALL | LCE_DW_BF16)) return LCE_ERR_INVALID_ARG;
    if (flags & LCE_INPUT_FP16) return LCE_ERR_UNSUPPORTED;
    const bool grad = dH != nullptr || dW != nullptr;
    const bool frozen = (flags & LCE_FROZEN_W) != 0 || !grad;
    const bool acc_dh = (flags & LCE_ACCUMULATE_DH) != 0, acc_dw0 = (flags & LCE_ACCUMULATE_DW) != 0;
    if ((flags & LCE_FROZEN_W) && acc_dw0) return LCE_ERR_INVALID_ARG;
    LCE_TRY(preference_check(offsets, pairs, ref_logprobs, beta, label_smoothing, reduction, dloss, loss,
                             seq_logprobs));
    if (grad && ((N > 0 && !dH) || (!frozen && !dW))) return LCE_ERR_INVALID_ARG;
    if ((dH && !aligned16(dH)) || (dW && !aligned16(dW))) return LCE_ERR_ALIGNMENT;
    if (grad) chunk = answer_chunk(N, chunk, flags);
    PrefLayout P;
    if (!make_pref_layout(N, D, V, chunk, pairs, flags, grad, P)) return LCE_ERR_INVALID_ARG;
    if (!ws) return LCE_ERR_INVALID_ARG;
    if (ws_bytes < P.total) return LCE_ERR_WORKSPACE;
    if ((flags & LCE_DW_BF16) && (frozen || acc_dw0 || P.L.nchunks > 1)) return LCE_ERR_UNSUPPORTED;
    const void *Hs = H;
    const int64_t *ys = y;
    LCE_TRY(gather_inputs(P.gather, Hs, ys, ws));
    Ctx c;
    LCE_TRY(setup(c, Hs, W, ys, N, D, V, ignore_index, chunk, ws, ws_bytes, stream, P.gather.on, false,
                  (flags & LCE_FROZEN_W) != 0, !grad, true, !P.gather.on, true));
    LCE_TRY(start_gather(c, P.gather, H, y));
    if (P.gather.on && grad && !acc_dh) LCE_ZERO(dH, 2 * static_cast<size_t>(N) * static_cast<size_t>(D));
    c.reduction = LCE_REDUCTION_NONE;   // (of the rows: each has a coefficient of its own)
    c.answers = true;
    c.dw16 = (flags & LCE_DW_BF16) != 0;
    if (grad) set_rests(c, P.gather, !frozen);
    c.zx = reinterpret_cast<float *>(c.ws + P.off_zx);
    c.fix = reinterpret_cast<float2 *>(c.ws + P.off_fix);
    float *lse = reinterpret_cast<float *>(c.ws + P.off_lse);
    float *coef = grad ? reinterpret_cast<float *>(c.ws + P.off_coef) : nullptr;
    if (frozen) dW = nullptr;
    const long long n = c.L.nchunks;
    if (n == 0 && dW && !acc_dw0 &&
        cudaMemsetAsync(dW, 0, (c.dw16 ? 2 : sizeof(float)) * static_cast<size_t>(V) * D, c.s) != cudaSuccess)
        return LCE_ERR_CUDA;
    for (long long i = 0; i < n; ++i) {
        const long long k = !grad || i + 1 < n ? (grad ? i + 1 : i) : 0;   // (with gradients the first chunk last)
        LCE_TRY(bring_rows(c, k, true));
        LCE_TRY(run_logits(c, grad && k == 0 ? MODE_LSE_P : MODE_LSE, k * c.L.C, chunk_rows(c, k), static_cast<int>(k),
                           nullptr, nullptr, c.Gb[0]));
        LCE_TRY(run_merge(c, k * c.L.C, chunk_rows(c, k), lse, nullptr, c.loss_rows));
    }
    PairParams pp = pair_params(offsets, pairs, N, V, ignore_index, y, c.loss_rows, ref_logprobs, beta, label_smoothing,
                                average, dloss, reduction, loss, seq_logprobs,
                                reinterpret_cast<float *>(c.ws + P.off_pair),
                                reinterpret_cast<int *>(c.ws + P.off_clean), coef, c.hdr);
    pp.fix = c.fix;
    pp.place = c.index ? reinterpret_cast<const int *>(c.ws + P.gather.off_place) : nullptr;
    if (pp.clean) LCE_LAUNCH(launch_offsets(pp, c.s));
    LCE_LAUNCH(launch_pairs(pp, c.s));
    if (!grad || n == 0) return LCE_OK;
    // the tile counters start again
    if (cudaMemsetAsync(c.hdr + HDR_COUNTERS, 0, c.L.hdr_bytes - sizeof(int) * HDR_COUNTERS, c.s) != cudaSuccess)
        return LCE_ERR_CUDA;
    c.coef = coef;
    __nv_bfloat16 *dHb = static_cast<__nv_bfloat16 *>(dH);
    const long long rows = chunk_rows(c, 0);
    LCE_TRY(run_prep(c, 0, rows, nullptr, coef, c.loss_rows, c.Gb[0], !frozen));
    LCE_TRY(run_grad(c, 0, rows, 1, dHb, acc_dh, dW, acc_dw0, coef,
                     GradSpec{c.Gb[0], c.Gb[0], frozen ? 0 : rows, true, false}));
    return backward_chunks(c, 1, n, lse, coef, dHb, acc_dh, dW, true);
}

lce_status lce_rmsnorm_forward(const void *X, const void *gamma, int64_t N, int64_t D, float eps,
                               void *H, float *rstd, lce_stream_t stream) {
    g_launches = 0;
    if (N < 0 || D <= 0 || D % 8 != 0 || D > NRM_MAX_D || !(eps >= 0.f)) return LCE_ERR_INVALID_ARG;
    if (N > 0 && (!X || !gamma || !H)) return LCE_ERR_INVALID_ARG;
    if ((X && !aligned16(X)) || (gamma && !aligned16(gamma)) || (H && !aligned16(H)))
        return LCE_ERR_ALIGNMENT;
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    NormParams p;
    memset(&p, 0, sizeof(p));
    p.X = static_cast<const __nv_bfloat16 *>(X);
    p.gamma = static_cast<const __nv_bfloat16 *>(gamma);
    p.H = static_cast<__nv_bfloat16 *>(H);
    p.rstd = rstd;
    p.rows = N;
    p.D = static_cast<int>(D);
    p.eps = eps;
    LCE_LAUNCH_KIND(LCE_KERNEL_NORM, s, launch_rmsnorm_fwd(p, s));
    return LCE_OK;
}

lce_status lce_rmsnorm_backward_workspace_size(int64_t D, size_t *bytes) {
    if (!bytes || D <= 0 || D % 8 != 0 || D > NRM_MAX_D) return LCE_ERR_INVALID_ARG;
    *bytes = align_up(4 * static_cast<size_t>(NRM_GRID) * static_cast<size_t>(D), 1024);
    return LCE_OK;
}

lce_status lce_rmsnorm_backward(const void *X, const void *gamma, const void *dH, int dh_fp32,
                                int64_t N, int64_t D, float eps, void *dX, float *dgamma, void *ws,
                                size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    size_t need = 0;
    if (lce_rmsnorm_backward_workspace_size(D, &need) != LCE_OK || N < 0 || !(eps >= 0.f))
        return LCE_ERR_INVALID_ARG;
    if (!gamma || !dgamma || !ws || (N > 0 && (!X || !dH || !dX))) return LCE_ERR_INVALID_ARG;
    if ((X && !aligned16(X)) || !aligned16(gamma) || (dH && !aligned16(dH)) ||
        (dX && !aligned16(dX)) || !aligned16(ws))
        return LCE_ERR_ALIGNMENT;
    if (ws_bytes < need) return LCE_ERR_WORKSPACE;
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    NormParams p;
    memset(&p, 0, sizeof(p));
    p.X = static_cast<const __nv_bfloat16 *>(X);
    p.gamma = static_cast<const __nv_bfloat16 *>(gamma);
    p.dH = dH;
    p.dh_fp32 = dh_fp32 ? 1 : 0;
    p.dX = static_cast<__nv_bfloat16 *>(dX);
    p.part = static_cast<float *>(ws);
    p.first = 1;
    p.rows = N;
    p.D = static_cast<int>(D);
    p.eps = eps;
    LCE_LAUNCH_KIND(LCE_KERNEL_NORM, s, launch_rmsnorm_bwd(p, s));
    LCE_LAUNCH_KIND(LCE_KERNEL_NORM, s, launch_dgamma_reduce(p.part, p.D, dgamma, s));
    return LCE_OK;
}

lce_status lce_norm_workspace_size_opt(int64_t N, int64_t D, int64_t V, int64_t chunk, int flags,
                                       size_t *bytes) {
    if (!bytes || (flags & ~(LCE_FROZEN_W | LCE_LOW_MEMORY))) return LCE_ERR_INVALID_ARG;
    NormLayout NL;
    if (!make_norm_layout(N, D, V, chunk, NL, (flags & LCE_FROZEN_W) != 0,
                          (flags & LCE_LOW_MEMORY) != 0))
        return LCE_ERR_INVALID_ARG;
    *bytes = NL.total;
    return LCE_OK;
}

lce_status lce_norm_workspace_size(int64_t N, int64_t D, int64_t V, int64_t chunk, size_t *bytes) {
    return lce_norm_workspace_size_opt(N, D, V, chunk, 0, bytes);
}

lce_status lce_norm_fwd_bwd_opt(const void *X, const void *gamma, float eps, const void *W,
                                const int64_t *y, const float *dloss, int64_t N, int64_t D,
                                int64_t V, int64_t ignore_index, int64_t chunk, int reduction,
                                int flags, float *loss, float *lse, void *dX, float *dgamma,
                                float *dW, void *ws, size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    if (flags & ~(LCE_FROZEN_W | LCE_LOW_MEMORY)) return LCE_ERR_INVALID_ARG;
    const bool frozen = (flags & LCE_FROZEN_W) != 0;
    const bool low_mem = (flags & LCE_LOW_MEMORY) != 0;
    const bool none = reduction == LCE_REDUCTION_NONE;
    NormLayout NL;
    if (!make_norm_layout(N, D, V, chunk, NL, frozen, low_mem) || !(eps >= 0.f))
        return LCE_ERR_INVALID_ARG;
    if (!gamma || !dgamma || (!frozen && !dW) || (!none && !loss) ||
        (N > 0 && (!X || !lse || !dX || !loss)))
        return LCE_ERR_INVALID_ARG;
    if ((X && !aligned16(X)) || !aligned16(gamma) || (dW && !aligned16(dW)) ||
        (dX && !aligned16(dX)) || (loss && !aligned16(loss)) || (lse && !aligned16(lse)))
        return LCE_ERR_ALIGNMENT;
    if (frozen) dW = nullptr;
    if (!ws) return LCE_ERR_INVALID_ARG;
    if (ws_bytes < NL.total) return LCE_ERR_WORKSPACE;
    uint8_t *w = static_cast<uint8_t *>(ws);
    __nv_bfloat16 *Hbuf = reinterpret_cast<__nv_bfloat16 *>(w + NL.off_H);
    float *dHbuf = reinterpret_cast<float *>(w + NL.off_dH);
    float *part = reinterpret_cast<float *>(w + NL.off_part);
    Ctx c;
    LCE_TRY(setup(c, Hbuf, W, y, N, D, V, ignore_index, chunk, ws, ws_bytes, stream, true, false,
                  frozen, false, low_mem || frozen));
    c.reduction = reduction;
    float *rows_out = none ? loss : c.loss_rows;
    if (c.L.nchunks == 0) {
        if ((dW && cudaMemsetAsync(dW, 0, sizeof(float) * static_cast<size_t>(V) * D, c.s) !=
                       cudaSuccess) ||
            cudaMemsetAsync(dgamma, 0, sizeof(float) * static_cast<size_t>(D), c.s) != cudaSuccess)
            return LCE_ERR_CUDA;
    }
    const __nv_bfloat16 *Xb = static_cast<const __nv_bfloat16 *>(X);
    __nv_bfloat16 *dXb = static_cast<__nv_bfloat16 *>(dX);
    const __nv_bfloat16 *gam = static_cast<const __nv_bfloat16 *>(gamma);
    // RMSNorm forward of rows [row0, row0 + rows) into their place in the H buffer
    auto norm_fwd = [&](long long row0, long long rows) -> lce_status {
        NormParams np;
        memset(&np, 0, sizeof(np));
        np.X = Xb + row0 * c.D;
        np.gamma = gam;
        np.H = Hbuf + h_row(c, row0) * c.D;
        np.rows = rows;
        np.D = static_cast<int>(c.D);
        np.eps = eps;
        LCE_LAUNCH_KIND(LCE_KERNEL_NORM, c.s, launch_rmsnorm_fwd(np, c.s));
        return LCE_OK;
    };
    // RMSNorm backward of a chunk from its fp32 dH (the sum of `parts` arrays)
    auto norm_bwd = [&](long long row0, long long rows, int parts) -> lce_status {
        NormParams np;
        memset(&np, 0, sizeof(np));
        np.X = Xb + row0 * c.D;
        np.gamma = gam;
        np.rows = rows;
        np.D = static_cast<int>(c.D);
        np.eps = eps;
        np.dH = dHbuf;
        np.dh_fp32 = 1;
        np.dh_splits = parts;
        np.dh_split_stride = c.L.ldp * c.D;
        np.dX = dXb + row0 * c.D;
        np.part = part;
        np.first = row0 == 0 ? 1 : 0;
        LCE_LAUNCH_KIND(LCE_KERNEL_NORM, c.s, launch_rmsnorm_bwd(np, c.s));
        return LCE_OK;
    };
    if (paired(c, true)) {
        // chunks in pairs (a, b), as on the loss path: the normalised rows of both
        // in the H buffer; a's logits, prep, a's dH tiles (fp32, in parts) with b's
        // logits beside them, a's RMSNorm backward; b's prep, b's dH beside one dW
        // contraction over both chunks, b's RMSNorm backward
        for (long long a = 0; a < c.L.nchunks; a += 2) {
            const long long ra = a * c.L.C, na = chunk_rows(c, a);
            const bool has_b = a + 1 < c.L.nchunks;
            const long long b = a + 1, rb = b * c.L.C, nb = has_b ? chunk_rows(c, b) : 0;
            LCE_TRY(norm_fwd(ra, na + nb));
            LCE_TRY(run_logits(c, MODE_LSE_P, ra, na, static_cast<int>(2 * a), nullptr, nullptr,
                               c.Gb[0]));
            LCE_TRY(run_prep(c, ra, na, lse, dloss, rows_out, c.Gb[0], true, 0));
            int parts = 1;
            if (!has_b) {
                LCE_TRY(run_bwd(c, ra, na, static_cast<int>(2 * a + 1),
                                DhOut{dHbuf, true, dh_parts(c, na, false), c.L.ldp}, dW, a > 0,
                                dloss, GradSpec{c.Gb[0], c.Gb[0], na, true, false}, &parts));
                LCE_TRY(norm_bwd(ra, na, parts));
                break;
            }
            const LogitsSpec lb{MODE_LSE_P, rb, nb, static_cast<int>(2 * b), nullptr, nullptr,
                                c.Gb[1]};
            GradSpec ga{c.Gb[0], c.Gb[0], 0, true, true};
            ga.beside = &lb;
            LCE_TRY(run_bwd(c, ra, na, static_cast<int>(2 * a + 1),
                            DhOut{dHbuf, true, dh_parts(c, na, true), c.L.ldp}, dW, false, dloss,
                            ga, &parts));
            LCE_TRY(norm_bwd(ra, na, parts));
            LCE_TRY(run_prep(c, rb, nb, lse, dloss, rows_out, c.Gb[1], true, c.L.C));
            LCE_TRY(run_bwd(c, rb, nb, static_cast<int>(2 * b + 1),
                            DhOut{dHbuf, true, dh_parts(c, nb, false), c.L.ldp}, dW, a > 0, dloss,
                            GradSpec{c.Gb[1], c.Gb[0], c.L.C + nb, true, false}, &parts));
            LCE_TRY(norm_bwd(rb, nb, parts));
        }
    } else {
        for (long long k = 0; k < c.L.nchunks; ++k) {
            const long long row0 = k * c.L.C;
            const long long rows = chunk_rows(c, k);
            LCE_TRY(norm_fwd(row0, rows));
            LCE_TRY(run_logits(c, MODE_LSE_P, row0, rows, static_cast<int>(2 * k), nullptr, nullptr,
                               c.Gb[0]));
            LCE_TRY(run_prep(c, row0, rows, lse, dloss, rows_out, c.Gb[0], !frozen));
            int parts = 1;
            LCE_TRY(run_bwd(c, row0, rows, static_cast<int>(2 * k + 1),
                            DhOut{dHbuf, true, dh_parts(c, rows, false), c.L.ldp}, dW, k > 0,
                            dloss, GradSpec{c.Gb[0], c.Gb[0], frozen ? 0 : rows, true, false},
                            &parts));
            LCE_TRY(norm_bwd(row0, rows, parts));
        }
    }
    if (!none)
        LCE_LAUNCH(launch_loss_finalize(c.loss_rows, c.N, c.hdr, loss,
                                        reduction == LCE_REDUCTION_MEAN, c.s));
    if (c.L.nchunks > 0)
        LCE_LAUNCH_KIND(LCE_KERNEL_NORM, c.s, launch_dgamma_reduce(part, static_cast<int>(c.D), dgamma, c.s));
    return LCE_OK;
}

lce_status lce_norm_fwd_bwd(const void *X, const void *gamma, float eps, const void *W,
                            const int64_t *y, const float *dloss, int64_t N, int64_t D, int64_t V,
                            int64_t ignore_index, int64_t chunk, int reduction, float *loss,
                            float *lse, void *dX, float *dgamma, float *dW, void *ws,
                            size_t ws_bytes, lce_stream_t stream) {
    return lce_norm_fwd_bwd_opt(X, gamma, eps, W, y, dloss, N, D, V, ignore_index, chunk, reduction,
                                0, loss, lse, dX, dgamma, dW, ws, ws_bytes, stream);
}

lce_status lce_ce_logits_workspace_size(int64_t N, size_t *bytes) {
    if (!bytes || N < 0) return LCE_ERR_INVALID_ARG;
    *bytes = 1024 + align_up(sizeof(float) * static_cast<size_t>(N > 0 ? N : 1), 1024);
    return LCE_OK;
}

lce_status lce_ce_logits(const void *Z, int z_dtype, int64_t ld, const int64_t *y, int64_t N,
                         int64_t V, int64_t ignore_index, int reduction, const float *dloss,
                         float *loss, float *lse, void *dZ, void *ws, size_t ws_bytes,
                         lce_stream_t stream) {
    g_launches = 0;
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    const bool none = reduction == LCE_REDUCTION_NONE;
    if (N < 0 || V <= 0 || ld < V || !ws) return LCE_ERR_INVALID_ARG;
    if (N > 0 && (!Z || !y || !lse || !loss)) return LCE_ERR_INVALID_ARG;
    if (!none && !loss) return LCE_ERR_INVALID_ARG;
    if (z_dtype < CE_BF16 || z_dtype > CE_FP16) return LCE_ERR_INVALID_ARG;
    const int vec = z_dtype == CE_FP32 ? 4 : 8;
    if (ld % vec != 0) return LCE_ERR_ALIGNMENT;
    if ((Z && !aligned16(Z)) || (dZ && !aligned16(dZ)) || !aligned16(ws) ||
        (loss && !aligned16(loss)) || (lse && !aligned16(lse)) || (y && !aligned16(y)))
        return LCE_ERR_ALIGNMENT;
    size_t need = 0;
    lce_ce_logits_workspace_size(N, &need);
    if (ws_bytes < need) return LCE_ERR_WORKSPACE;
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *w = static_cast<uint8_t *>(ws);
    int *hdr = reinterpret_cast<int *>(w);
    float *loss_rows = reinterpret_cast<float *>(w + 1024);
    if (cudaMemsetAsync(hdr, 0, 1024, s) != cudaSuccess) return LCE_ERR_CUDA;
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s,
                    launch_label_scan(reinterpret_cast<const long long *>(y), N, V, ignore_index, hdr, s));
    CELogitsParams p;
    p.Z = Z;
    p.dZ = dZ;
    p.ld = ld;
    p.dtype = z_dtype;
    p.N = N;
    p.V = V;
    p.ignore_index = ignore_index;
    p.y = reinterpret_cast<const long long *>(y);
    p.hdr = hdr;
    p.dloss = dloss;
    p.dloss_per_row = none ? 1 : 0;
    p.mean = reduction == LCE_REDUCTION_MEAN ? 1 : 0;
    p.lse = lse;
    p.loss_rows = none ? loss : loss_rows;
    LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, s, launch_ce_logits(p, sms, s));
    if (!none)
        LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s,
                        launch_loss_finalize(loss_rows, N, hdr, loss,
                                             reduction == LCE_REDUCTION_MEAN, s));
    return LCE_OK;
}

namespace {

// Checks that both losses over logits share; the element size.
lce_status answer_logits_check(const void *Z, int z_dtype, int64_t ld, const int64_t *y, int64_t N, int64_t V,
                               const float *dloss, const float *loss, const void *dZ, const void *ws) {
    if (N < 0 || N > 0x7fffffffll || V <= 0 || V > MAX_V || ld < V || !ws) return LCE_ERR_INVALID_ARG;
    if (z_dtype < CE_BF16 || z_dtype > CE_FP16 || (N > 0 && (!Z || !y))) return LCE_ERR_INVALID_ARG;
    const uintptr_t z = reinterpret_cast<uintptr_t>(Z), d = reinterpret_cast<uintptr_t>(dZ);
    if (z % (z_dtype == CE_FP32 ? 4 : 2) || reinterpret_cast<uintptr_t>(y) % 8 || !aligned16(ws) ||
        (reinterpret_cast<uintptr_t>(dloss) | reinterpret_cast<uintptr_t>(loss)) % 4)
        return LCE_ERR_ALIGNMENT;
    if (dZ && z % 16 != d % 16) return LCE_ERR_ALIGNMENT;
    // dZ is Z, or lies beside it
    const uintptr_t bytes = N > 0 ? ((static_cast<uintptr_t>(N) - 1) * ld + V) * (z_dtype == CE_FP32 ? 4 : 2) : 0;
    if (dZ && d != z && d < z + bytes && z < d + bytes) return LCE_ERR_INVALID_ARG;
    return LCE_OK;
}

AnswerParams answer_params(const void *Z, int z_dtype, int64_t ld, const int64_t *y, int64_t N, int64_t V,
                           int64_t ign, int *hdr) {
    AnswerParams p;
    memset(&p, 0, sizeof(p));
    p.Z = Z;
    p.ld = ld;
    p.dtype = z_dtype;
    p.N = N;
    p.V = V;
    p.ignore_index = ign;
    p.y = reinterpret_cast<const long long *>(y);
    p.hdr = hdr;
    p.pol.inv_t = 1.f;
    return p;
}

}  // namespace

lce_status lce_policy_logits(const void *Z, int z_dtype, int64_t ld, const int64_t *y, const float *advantages,
                             const float *old_logprobs, const float *ref_logprobs, const float *weights,
                             float clip_low, float clip_high, float beta, float temperature, const float *dloss,
                             int64_t N, int64_t V, int64_t ignore_index, int reduction, float *loss,
                             float *logprobs, void *dZ, void *ws, size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    if (reduction < LCE_REDUCTION_MEAN || reduction > LCE_REDUCTION_NONE) return LCE_ERR_INVALID_ARG;
    const bool none = reduction == LCE_REDUCTION_NONE;
    if (!loss && (N > 0 || !none)) return LCE_ERR_INVALID_ARG;
    LCE_TRY(policy_check(N, advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta,
                         temperature, logprobs));
    LCE_TRY(answer_logits_check(Z, z_dtype, ld, y, N, V, dloss, loss, dZ, ws));
    size_t need = 0;
    lce_ce_logits_workspace_size(N, &need);
    if (ws_bytes < need) return LCE_ERR_WORKSPACE;
    int sms = 0, pairs = 0;
    LCE_TRY(init_device(&sms, &pairs));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *w = static_cast<uint8_t *>(ws);
    AnswerParams p = answer_params(Z, z_dtype, ld, y, N, V, ignore_index, reinterpret_cast<int *>(w));
    p.dZ = dZ;
    p.dloss = dloss;
    p.dloss_per_row = none ? 1 : 0;
    p.mean = reduction == LCE_REDUCTION_MEAN ? 1 : 0;
    p.pol = policy_params(advantages, old_logprobs, ref_logprobs, weights, clip_low, clip_high, beta, temperature,
                          logprobs);
    p.loss_rows = none ? loss : reinterpret_cast<float *>(w + 1024);
    p.loss = none ? nullptr : loss;
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_answer_scan(p.y, N, V, ignore_index, p.hdr, s));
    if (N > 0) LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, s, launch_answer_rows(p, sms, s));
    else if (loss && cudaMemsetAsync(loss, 0, sizeof(float), s) != cudaSuccess) return LCE_ERR_CUDA;
    return LCE_OK;
}

lce_status lce_preference_logits_workspace_size(int64_t N, int64_t pairs, size_t *bytes) {
    if (!bytes || N < 0 || N > 0x7fffffffll || pairs <= 0 || pairs > (1ll << 24)) return LCE_ERR_INVALID_ARG;
    const size_t rows = align_up(sizeof(float) * static_cast<size_t>(N > 0 ? N : 1), 1024);
    *bytes = 1024 + 4 * rows + align_up(sizeof(float) * static_cast<size_t>(pairs), 1024) +
             align_up(sizeof(int) * static_cast<size_t>(2 * pairs + 1), 1024);
    return LCE_OK;
}

lce_status lce_preference_logits(const void *Z, int z_dtype, int64_t ld, const int64_t *y, const int64_t *offsets,
                                 int64_t pairs_, const float *ref_logprobs, float beta, float label_smoothing,
                                 int average, const float *dloss, int64_t N, int64_t V, int64_t ignore_index,
                                 int reduction, float *loss, float *seq_logprobs, void *dZ, void *ws,
                                 size_t ws_bytes, lce_stream_t stream) {
    g_launches = 0;
    LCE_TRY(preference_check(offsets, pairs_, ref_logprobs, beta, label_smoothing, reduction, dloss, loss,
                             seq_logprobs));
    LCE_TRY(answer_logits_check(Z, z_dtype, ld, y, N, V, dloss, loss, dZ, ws));
    size_t need = 0;
    LCE_TRY(lce_preference_logits_workspace_size(N, pairs_, &need));
    if (ws_bytes < need) return LCE_ERR_WORKSPACE;
    int sms = 0, pairs = 0;
    LCE_TRY(init_device(&sms, &pairs));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *w = static_cast<uint8_t *>(ws);
    const size_t rows = align_up(sizeof(float) * static_cast<size_t>(N > 0 ? N : 1), 1024);
    AnswerParams p = answer_params(Z, z_dtype, ld, y, N, V, ignore_index, reinterpret_cast<int *>(w));
    p.loss_rows = reinterpret_cast<float *>(w + 1024);
    float *coef = reinterpret_cast<float *>(w + 1024 + rows);
    p.max_sum = reinterpret_cast<float2 *>(w + 1024 + 2 * rows);
    float *pair_loss = reinterpret_cast<float *>(w + 1024 + 4 * rows);
    int *clean = reinterpret_cast<int *>(w + 1024 + 4 * rows + align_up(sizeof(float) * static_cast<size_t>(pairs_), 1024));
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_answer_scan(p.y, N, V, ignore_index, p.hdr, s));
    if (N > 0) LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, s, launch_answer_rows(p, sms, s));
    const PairParams pp = pair_params(offsets, pairs_, N, V, ignore_index, y, p.loss_rows, ref_logprobs, beta,
                                      label_smoothing, average, dloss, reduction, loss, seq_logprobs, pair_loss, clean,
                                      dZ ? coef : nullptr, p.hdr);
    if (pp.clean) LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_offsets(pp, s));
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_pairs(pp, s));
    if (dZ && N > 0) {
        p.dZ = dZ;
        p.coef = coef;
        LCE_LAUNCH_KIND(LCE_KERNEL_MERGE, s, launch_answer_grad(p, sms, s));
    }
    return LCE_OK;
}

lce_status lce_scale(const void *src, int src_dtype, const float *scale, int64_t n, void *dst, int dst_dtype,
                     lce_stream_t stream) {
    g_launches = 0;
    if (n < 0 || src_dtype < CE_BF16 || src_dtype > CE_FP16 || dst_dtype < CE_BF16 || dst_dtype > CE_FP16 ||
        !scale || (n > 0 && (!src || !dst)))
        return LCE_ERR_INVALID_ARG;
    const uintptr_t a = reinterpret_cast<uintptr_t>(src), b = reinterpret_cast<uintptr_t>(dst);
    const uintptr_t ea = src_dtype == CE_FP32 ? 4 : 2, eb = dst_dtype == CE_FP32 ? 4 : 2;
    if (a % ea || b % eb || reinterpret_cast<uintptr_t>(scale) % 4) return LCE_ERR_ALIGNMENT;
    if (n > 0 && !(a == b && src_dtype == dst_dtype) && a < b + eb * n && b < a + ea * n) return LCE_ERR_INVALID_ARG;
    int sms = 0, pairs = 0;
    LCE_TRY(init_device(&sms, &pairs));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n > 0) LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_scale(src, src_dtype, scale, n, dst, dst_dtype, sms, s));
    return LCE_OK;
}

lce_status lce_sample_logits(const void *Z, int z_dtype, int64_t ld, int64_t N, int64_t V,
                             const float *u, const float *temperature, const int32_t *top_k,
                             const float *top_p, const float *min_p, float temperature_all,
                             int32_t top_k_all, float top_p_all, float min_p_all,
                             int64_t *tokens, float *logprobs, lce_stream_t stream) {
    g_launches = 0;
    if (N < 0 || N > (1ll << 27) || V <= 0 || V > SMP_MAX_V || ld < V) return LCE_ERR_INVALID_ARG;
    if (z_dtype < CE_BF16 || z_dtype > CE_FP16) return LCE_ERR_INVALID_ARG;
    if (N > 0 && (!Z || !u || !tokens)) return LCE_ERR_INVALID_ARG;
    const uintptr_t elem = z_dtype == CE_FP32 ? 4 : 2;
    const uintptr_t words = reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(temperature) |
                            reinterpret_cast<uintptr_t>(top_k) | reinterpret_cast<uintptr_t>(top_p) |
                            reinterpret_cast<uintptr_t>(min_p) | reinterpret_cast<uintptr_t>(logprobs);
    if (reinterpret_cast<uintptr_t>(Z) % elem || words % 4 || reinterpret_cast<uintptr_t>(tokens) % 8)
        return LCE_ERR_ALIGNMENT;
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    if (N == 0) return LCE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    SampleParams p;
    p.Z = Z;
    p.ld = ld;
    p.N = N;
    p.V = static_cast<int>(V);
    p.dtype = z_dtype;
    p.u = u;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.temperature_all = temperature_all;
    p.top_k_all = top_k_all;
    p.top_p_all = top_p_all;
    p.min_p_all = min_p_all;
    p.tokens = reinterpret_cast<long long *>(tokens);
    p.logprobs = logprobs;
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_sample(p, sms, s));
    return LCE_OK;
}

lce_status lce_fp8_quantize(const void *X, int x_dtype, int64_t ld, int64_t R, int64_t C, int tiles,
                            void *q, int64_t ldq, float *scale, void *qt, int64_t ldqt,
                            float *scale_t, lce_stream_t stream) {
    g_launches = 0;
    if (x_dtype < CE_BF16 || x_dtype > CE_FP16) return LCE_ERR_INVALID_ARG;
    if (R < 0 || C <= 0 || R > 0x7fffffffll || C > 0x7fffffffll || ld < C) return LCE_ERR_INVALID_ARG;
    if ((!q && !qt) || (R > 0 && !X)) return LCE_ERR_INVALID_ARG;
    if ((q && (!scale || ldq < C)) || (qt && (!scale_t || ldqt < R))) return LCE_ERR_INVALID_ARG;
    const uintptr_t elem = x_dtype == CE_FP32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(X) % elem || (q && (!aligned16(q) || ldq % 16)) ||
        (qt && (!aligned16(qt) || ldqt % 16)) || reinterpret_cast<uintptr_t>(scale) % 4 ||
        reinterpret_cast<uintptr_t>(scale_t) % 4)
        return LCE_ERR_ALIGNMENT;
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    Fp8QuantParams p;
    p.X = X;
    p.ld = ld;
    p.R = R;
    p.C = C;
    p.rblocks = cdiv(R, 128);
    p.cblocks = cdiv(C, 128);
    if (p.rblocks * p.cblocks > 0x7fffffffll) return LCE_ERR_INVALID_ARG;
    p.vec = aligned16(X) && (ld * static_cast<int64_t>(elem)) % 16 == 0 ? 1 : 0;
    p.q = static_cast<uint8_t *>(q);
    p.ldq = ldq;
    p.scale = scale;
    p.qt = static_cast<uint8_t *>(qt);
    p.ldqt = ldqt;
    p.scale_t = scale_t;
    if (R == 0) return LCE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_fp8_quantize(p, x_dtype, tiles != 0, s));
    return LCE_OK;
}

lce_status lce_fp8_matmul_workspace_size(size_t *bytes) {
    if (!bytes) return LCE_ERR_INVALID_ARG;
    *bytes = 1024;
    return LCE_OK;
}

lce_status lce_fp8_matmul(const void *A, int64_t lda, const float *sa, int64_t sa_row,
                          int64_t sa_block, const void *B, int64_t ldb, const float *sb,
                          int64_t sb_row, int64_t sb_block, int b_rows, int64_t M, int64_t N,
                          int64_t K, void *out, int64_t ldc, int c_dtype, void *ws, size_t ws_bytes,
                          lce_stream_t stream) {
    g_launches = 0;
    return fp8_matmul(A, lda, sa, sa_row, sa_block, B, ldb, sb, sb_row, sb_block, b_rows, M, N, K, out,
                      ldc, c_dtype, ws, ws_bytes, static_cast<uint8_t *>(ws) + 1024,
                      ws_bytes > 1024 ? ws_bytes - 1024 : 0, false, stream);
}

lce_status lce_fp8_matmul_best_workspace_size(int64_t M, int64_t N, int64_t K, int b_rows, size_t *bytes) {
    if (!bytes || M < 0 || N < 0 || K <= 0 || M > MAX_V || N > MAX_V || K > MAX_V) return LCE_ERR_INVALID_ARG;
    int sms = 0, pairs = 0;
    const lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    *bytes = 1024;
    if (!b_rows && fp8_pairs(M, N, sms, pairs))
        *bytes += fp8_parts_bytes(M, N, fp8_parts(cdiv(M, 256) * cdiv(N, 256), M, N, cdiv(K, 128), pairs));
    return LCE_OK;
}
lce_status lce_fp8_linear_workspace_size(int64_t M, int64_t K, size_t *bytes) {
    if (!bytes || M < 0 || K <= 0 || M > MAX_V || K > MAX_V) return LCE_ERR_INVALID_ARG;
    *bytes = 1024 + align_up(sizeof(float) * static_cast<size_t>(M) * cdiv(K, 128), 1024) +
             static_cast<size_t>(M) * align_up(static_cast<size_t>(K), 16);
    return LCE_OK;
}

lce_status lce_fp8_linear(const void *X, int x_dtype, int64_t ldx, const void *W, int64_t ldw,
                          const float *sw, int64_t sw_row, int64_t sw_block, int64_t M, int64_t N,
                          int64_t K, void *out, int64_t ldc, int c_dtype, void *ws, size_t ws_bytes,
                          lce_stream_t stream) {
    g_launches = 0;
    size_t need = 0;
    lce_status st = lce_fp8_linear_workspace_size(M, K, &need);
    if (st != LCE_OK) return st;
    if (!ws) return LCE_ERR_INVALID_ARG;
    if (!aligned16(ws)) return LCE_ERR_ALIGNMENT;
    if (ws_bytes < need) return LCE_ERR_WORKSPACE;
    uint8_t *w = static_cast<uint8_t *>(ws);
    float *sx = reinterpret_cast<float *>(w + 1024);
    uint8_t *xq = w + 1024 + align_up(sizeof(float) * static_cast<size_t>(M) * cdiv(K, 128), 1024);
    const int64_t ldq = static_cast<int64_t>(align_up(static_cast<size_t>(K), 16));
    // (the product's arguments are checked before the quantisation is enqueued)
    st = fp8_matmul_check(xq, ldq, sx, 1, M, W, ldw, sw, sw_row, sw_block, M, N, K, out, ldc, c_dtype, ws, ws_bytes);
    if (st != LCE_OK) return st;
    st = lce_fp8_quantize(X, x_dtype, ldx, M, K, 0, xq, ldq, sx, nullptr, 0, nullptr, stream);
    if (st != LCE_OK) return st;
    // (sums of parts lie behind X, which the product is reading)
    const size_t behind = align_up(need, 1024);
    return fp8_matmul(xq, ldq, sx, 1, M, W, ldw, sw, sw_row, sw_block, 0, M, N, K, out, ldc, c_dtype, ws, ws_bytes,
                      w + behind, ws_bytes > behind ? ws_bytes - behind : 0, M > 0, stream);
}

lce_status lce_int4_quantize(const void *W, int w_dtype, int64_t ldw, int64_t V, int64_t D, int group, void *q,
                             int64_t ldq, void *scale, int scale_dtype, int64_t lds, lce_stream_t stream) {
    g_launches = 0;
    if (w_dtype < CE_BF16 || w_dtype > CE_FP16 || (scale_dtype != CE_BF16 && scale_dtype != CE_FP16))
        return LCE_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return LCE_ERR_INVALID_ARG;
    if (V < 0 || V > 0x7fffffffll || D <= 0 || D > I4_MAX_D || ldw < D || ldq < (D + 31) / 32 * 16 ||
        lds < cdiv(D, group))
        return LCE_ERR_INVALID_ARG;
    if (V > 0 && (!W || !q || !scale)) return LCE_ERR_INVALID_ARG;
    if (ldq % 16 || !aligned16(q) || reinterpret_cast<uintptr_t>(W) % (w_dtype == CE_FP32 ? 4 : 2) ||
        reinterpret_cast<uintptr_t>(scale) % 2)
        return LCE_ERR_ALIGNMENT;
    int sms = 0, pairs = 0;
    LCE_TRY(init_device(&sms, &pairs));
    if (V == 0) return LCE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Int4QuantParams p;
    p.W = W;
    p.ldw = ldw;
    p.V = V;
    p.D = static_cast<int>(D);
    p.dtype = w_dtype;
    p.group = group;
    p.q = static_cast<uint8_t *>(q);
    p.ldq = ldq;
    p.scale = scale;
    p.lds = lds;
    p.scale_dtype = scale_dtype;
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_int4_quantize(p, s));
    return LCE_OK;
}

lce_status lce_int4_linear_workspace_size(int64_t M, int64_t D, int group, size_t *bytes) {
    if (!bytes || M < 0 || M > (1ll << 20) || D <= 0 || D > I4_MAX_D) return LCE_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return LCE_ERR_INVALID_ARG;
    *bytes = M == 0 || int4_few(M, D, group)
                 ? 0
                 : 1024 + align_up(4 * static_cast<size_t>(M), 1024) +
                       static_cast<size_t>(M) * static_cast<size_t>(cdiv(D, 128)) * 256;
    return LCE_OK;
}

namespace {

// bring: false for the self-test, whose waits run out after limit_ns.
lce_status int4_linear(const void *X, int x_dtype, int64_t ldx, const void *q, int64_t ldq, const void *scale,
                       int64_t lds, int group, int64_t M, int64_t V, int64_t D, void *out, int64_t ldc, void *ws,
                       size_t ws_bytes, bool bring, unsigned long long limit_ns, lce_stream_t stream) {
    g_launches = 0;
    if (x_dtype != CE_BF16 && x_dtype != CE_FP16) return LCE_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return LCE_ERR_INVALID_ARG;
    if (M < 0 || M > (1ll << 20) || V <= 0 || V > MAX_V || D <= 0 || D > I4_MAX_D || ldx < D || ldc < V ||
        ldq < (D + 31) / 32 * 16 || lds < cdiv(D, group))
        return LCE_ERR_INVALID_ARG;
    size_t need = 0;
    LCE_TRY(lce_int4_linear_workspace_size(M, D, group, &need));
    if (!q || !scale || (need && !ws) || (M > 0 && (!X || !out))) return LCE_ERR_INVALID_ARG;
    const uintptr_t halves = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(scale) |
                             reinterpret_cast<uintptr_t>(out);
    if (ldq % 16 || !aligned16(q) || halves % 2 || !aligned16(ws)) return LCE_ERR_ALIGNMENT;
    if (ws_bytes < need) return LCE_ERR_WORKSPACE;
    int sms = 0, pairs = 0;
    LCE_TRY(init_device(&sms, &pairs));
    if (M == 0) return LCE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int x_vec = aligned16(X) && ldx % 8 == 0;
    if (int4_few(M, D, group)) {
        Int4Params p;
        p.X = X;
        p.ldx = ldx;
        p.dtype = x_dtype;
        p.x_vec = x_vec;
        p.q = static_cast<const uint8_t *>(q);
        p.ldq = ldq;
        p.scale = scale;
        p.lds = lds;
        p.group = group;
        p.M = static_cast<int>(M);
        p.V = static_cast<int>(V);
        p.D = static_cast<int>(D);
        p.out = out;
        p.ldc = ldc;
        LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_int4(p, sms, s));
        return LCE_OK;
    }
    uint8_t *w = static_cast<uint8_t *>(ws);
    Int4TileParams p;
    memset(&p, 0, sizeof(p));
    const int n = int4_tile_tokens(M);
    p.scale = scale;
    p.lds = lds;
    p.hdr = reinterpret_cast<int *>(w);
    p.down = reinterpret_cast<float *>(w + 1024);
    void *tokens = w + 1024 + align_up(4 * static_cast<size_t>(M), 1024);
    p.out = out;
    p.ldc = ldc;
    p.dtype = x_dtype;
    p.M = static_cast<int>(M);
    p.V = static_cast<int>(V);
    p.D = static_cast<int>(D);
    p.units = static_cast<int>(cdiv(D, 128));
    p.groups = static_cast<int>(cdiv(D, group));
    p.per = 128 / group;
    p.row_tiles = static_cast<int>(cdiv(V, 128));
    p.token_tiles = static_cast<int>(cdiv(M, n));
    if (static_cast<long long>(p.row_tiles) * p.token_tiles > 0x7fffffffll) return LCE_ERR_INVALID_ARG;
    p.bring = bring ? 1 : 0;
    p.timeout_ns = limit_ns;
    const uint64_t dims[2] = {static_cast<uint64_t>((D + 31) / 32 * 16), static_cast<uint64_t>(V)};
    const uint64_t st[1] = {static_cast<uint64_t>(ldq)};
    const uint32_t box[2] = {128, 128};
    if (!encode_map(&p.tmQ, q, 2, dims, st, box, MAP_U8)) return LCE_ERR_CUDA;
    if (!encode_2d(&p.tmX, tokens, static_cast<uint64_t>(p.units) * 128, M, static_cast<uint64_t>(p.units) * 256, 64,
                   static_cast<uint32_t>(n), MAP_F16))
        return LCE_ERR_CUDA;
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_int4_tokens(p, X, ldx, x_vec, tokens, s));
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s, launch_int4_tiles(p, n, sms, s));
    return LCE_OK;
}

}  // namespace

lce_status lce_int4_linear(const void *X, int x_dtype, int64_t ldx, const void *q, int64_t ldq, const void *scale,
                           int64_t lds, int group, int64_t M, int64_t V, int64_t D, void *out, int64_t ldc,
                           void *ws, size_t ws_bytes, lce_stream_t stream) {
    return int4_linear(X, x_dtype, ldx, q, ldq, scale, lds, group, M, V, D, out, ldc, ws, ws_bytes, true,
                       kDefaultTimeoutNs, stream);
}

lce_status lce_selftest_int4_timeout(const void *X, int x_dtype, int64_t ldx, const void *q, int64_t ldq,
                                     const void *scale, int64_t lds, int group, int64_t M, int64_t V, int64_t D,
                                     void *out, int64_t ldc, void *ws, size_t ws_bytes, int64_t limit_us,
                                     lce_stream_t stream) {
    if (limit_us < 1 || limit_us > 2000000) return LCE_ERR_INVALID_ARG;
    size_t need = 0;
    LCE_TRY(lce_int4_linear_workspace_size(M, D, group, &need));
    if (need == 0) return LCE_ERR_INVALID_ARG;
    return int4_linear(X, x_dtype, ldx, q, ldq, scale, lds, group, M, V, D, out, ldc, ws, ws_bytes, false,
                       static_cast<unsigned long long>(limit_us) * 1000ull, stream);
}

lce_status lce_grad_norm_workspace_size(int64_t n, size_t *bytes) {
    if (!bytes || n < 0 || n > kMaxGrads) return LCE_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(n > 0 ? cdiv(n, CLIP_MAX_TENSORS) : 1) * CLIP_MAX_PARTS * sizeof(double);
    return LCE_OK;
}

lce_status lce_grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                         int64_t n, int norm_kind, float *norm, void *ws, size_t ws_bytes,
                         lce_stream_t stream) {
    return grad_norm(grads, sizes, dtypes, nullptr, n, norm_kind, false, 0.f, 0.f, norm, ws, ws_bytes,
                     stream);
}

lce_status lce_clip_grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                              void *const *outs, int64_t n, int norm_kind, float max_norm, float eps,
                              float *norm, void *ws, size_t ws_bytes, lce_stream_t stream) {
    if (!(max_norm >= 0.f) || !(eps >= 0.f)) {
        g_launches = 0;
        return LCE_ERR_INVALID_ARG;
    }
    return grad_norm(grads, sizes, dtypes, outs, n, norm_kind, true, max_norm, eps, norm, ws, ws_bytes,
                     stream);
}

lce_status lce_selftest_wait_timeout(void *ws, size_t ws_bytes, int64_t limit_us,
                                     lce_stream_t stream) {
    g_launches = 0;
    if (!ws || ws_bytes < 1024) return LCE_ERR_INVALID_ARG;
    if (limit_us < 1 || limit_us > 2000000) return LCE_ERR_INVALID_ARG;
    if (!aligned16(ws)) return LCE_ERR_ALIGNMENT;
    int sms = 0, pairs = 0;
    lce_status st = init_device(&sms, &pairs);
    if (st != LCE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(ws, 0, 1024, s) != cudaSuccess) return LCE_ERR_CUDA;
    LCE_LAUNCH_KIND(LCE_KERNEL_OTHER, s,
                    launch_wait_selftest(static_cast<int *>(ws),
                                         static_cast<unsigned long long>(limit_us) * 1000ull, s));
    return LCE_OK;
}

lce_status lce_read_status(const void *ws, lce_stream_t stream) {
    if (!ws) return LCE_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return LCE_ERR_CUDA;
    int flag = 0;
    if (cudaMemcpy(&flag, ws, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return LCE_ERR_CUDA;
    if (flag) {
        const int zero = 0;
        if (cudaMemcpy(const_cast<void *>(ws), &zero, sizeof(int), cudaMemcpyHostToDevice) !=
            cudaSuccess)
            return LCE_ERR_CUDA;
    }
    if (flag & FLAG_TIMEOUT) return LCE_ERR_TIMEOUT;
    if (flag & FLAG_OFFSETS) return LCE_ERR_OFFSETS;
    if (flag & FLAG_LABEL) return LCE_ERR_LABEL_RANGE;
    return LCE_OK;
}

const char *lce_status_string(lce_status s) {
    switch (s) {
        case LCE_OK: return "ok";
        case LCE_ERR_INVALID_ARG: return "invalid argument";
        case LCE_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
        case LCE_ERR_WORKSPACE: return "workspace too small";
        case LCE_ERR_LABEL_RANGE: return "label outside [0, V) and not ignore_index";
        case LCE_ERR_TIMEOUT: return "device pipeline wait timed out";
        case LCE_ERR_CUDA: return "CUDA runtime error";
        case LCE_ERR_UNSUPPORTED: return "device is not sm_103";
        case LCE_ERR_OFFSETS: return "offsets of sequences decrease or leave the rows";
    }
    return "unknown status";
}

int lce_version(void) { return 100; }

int lce_last_launch_count(void) { return g_launches; }

lce_status lce_profile_enable(int on) {
    std::lock_guard<std::mutex> lock(g_prof_mu);
    g_prof_on = on != 0;
    return LCE_OK;
}

lce_status lce_profile_read(int kind, double *total_ms, int64_t *launches) {
    if (kind < 0 || kind >= LCE_KERNEL_KINDS || !total_ms || !launches) return LCE_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(g_prof_mu);
    for (ProfPair &p : g_prof_pending) {
        if (cudaEventSynchronize(p.b) != cudaSuccess) return LCE_ERR_CUDA;
        float ms = 0.f;
        if (cudaEventElapsedTime(&ms, p.a, p.b) != cudaSuccess) return LCE_ERR_CUDA;
        g_prof_ms[p.kind] += ms;
        g_prof_n[p.kind] += 1;
        g_prof_pool.push_back(p.a);
        g_prof_pool.push_back(p.b);
    }
    g_prof_pending.clear();
    *total_ms = g_prof_ms[kind];
    *launches = g_prof_n[kind];
    return LCE_OK;
}

void lce_profile_reset(void) {
    std::lock_guard<std::mutex> lock(g_prof_mu);
    for (int k = 0; k < LCE_KERNEL_KINDS; ++k) {
        g_prof_ms[k] = 0.0;
        g_prof_n[k] = 0;
    }
}

}  // extern "C"
