// Host side of the layer operators (include/layer_ops.h): argument checks,
// tensor maps, workspaces and launches.  Part of the library's one translation
// unit (tcgemm.cu), behind gemm_f16.cu, whose device facts, tuning config and
// status word it shares.
#pragma once

#include "layer_ops.h"

#include "grad_clip_kernel.cuh"
#include "layer_grads_kernel.cuh"
#include "layer_pair_kernel.cuh"
#include "layer_skinny_kernel.cuh"
#include "layer_small_kernels.cuh"

namespace {

constexpr long long kMaxDim = INT_MAX - 1024;

// One matrix as the caller describes it.
struct Mat {
    const void* p;
    long long rows, cols, ld;
    int bytes;  // of an element
};

Mat mat16(const void* p, long long rows, long long cols, long long ld) { return Mat{p, rows, cols, ld, 2}; }

bool empty(const Mat& m) { return m.rows == 0 || m.cols == 0; }

// Bytes from the first to one past the last element.
uint64_t extent(const Mat& m) { return ((uint64_t)(m.rows - 1) * m.ld + m.cols) * m.bytes; }

int check_mat(const Mat& m) {
    if (empty(m)) return GEMM_OK;
    if (!m.p) return GEMM_ERR_NULL;
    // a tensor map's row stride stays below 2^40 bytes (in elements first: the product may overflow)
    if (m.ld < m.cols || m.ld >= (1ll << 40) / m.bytes) return GEMM_ERR_DIM;
    if (((uintptr_t)m.p & 15) || (m.ld * m.bytes) % 16 != 0) return GEMM_ERR_ALIGN;
    return GEMM_OK;
}

// Bytes [lo, hi), of which a matrix with a row stride takes `width` every `stride`.
struct Span {
    uint64_t lo, hi, stride, width;
};

Span span_of(const Mat& m) {
    if (!m.p || empty(m)) return Span{0, 0};
    return Span{(uint64_t)(uintptr_t)m.p, (uint64_t)(uintptr_t)m.p + extent(m), (uint64_t)m.ld * m.bytes,
                (uint64_t)m.cols * m.bytes};
}

Span span_of(const void* p, uint64_t bytes) {
    if (!p || bytes == 0) return Span{0, 0};
    return Span{(uint64_t)(uintptr_t)p, (uint64_t)(uintptr_t)p + bytes};
}

// Whether any of the `nw` written spans overlaps another of them or a read one.  Column
// ranges of the same rows (one stride) may lie side by side.
bool overlaps(const Span* w, int nw, const Span* r, int nr) {
    auto meet = [](const Span& a, const Span& b) {
        if (a.lo >= b.hi || b.lo >= a.hi) return false;
        if (a.stride == 0 || a.stride != b.stride) return true;
        const uint64_t gap = b.lo >= a.lo ? (b.lo - a.lo) % a.stride : a.stride - (a.lo - b.lo) % a.stride;
        return gap < a.width || gap + b.width > a.stride;
    };
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (meet(w[i], w[j])) return true;
        for (int j = 0; j < nr; ++j)
            if (meet(w[i], r[j])) return true;
    }
    return false;
}

bool dims_ok(std::initializer_list<long long> positive, long long tokens) {
    if (tokens < 0 || tokens > kMaxDim) return false;
    for (long long d : positive)
        if (d < 1 || d > kMaxDim) return false;
    return true;
}

int check_dtype_act(long long dtype, long long act) {
    if (dtype != LAYER_F16 && dtype != LAYER_BF16) return GEMM_ERR_DTYPE;
    if (act < LAYER_ACT_NONE || act > LAYER_ACT_GELU_TANH) return GEMM_ERR_CONFIG;
    return GEMM_OK;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
long long pad8(long long n) { return (n + 7) & ~7ll; }

// What a call needs of the current device, once its arguments are checked.
struct Ctx {
    DeviceInfo* dev = nullptr;
    int ordinal = 0;
    long long wait_limit = 0;
    int inject = 0;
    cudaStream_t stream = nullptr;
};

int open_ctx(Ctx& c, gemm_stream_t stream) {
    const gemm_config cfg = current_config();
    const int rc = device_info(&c.dev);
    if (rc != GEMM_OK) return rc;
    if (c.dev->cc != 103) return GEMM_ERR_ARCH;
    std::call_once(g_encode_once, init_encode);
    if (!g_encode) return GEMM_ERR_CUDA;
    c.ordinal = (int)(c.dev - g_dev);
    c.wait_limit = cfg.wait_limit > 0 ? cfg.wait_limit : kDefaultWaitLimit;
    c.inject = cfg.inject_stall;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return GEMM_OK;
}

// A 128-byte-swizzled tensor map of a matrix with a row stride; outside the
// matrix it reads zero and writes nothing.
int encode_mat(CUtensorMap* out, const Mat& m, int dtype, uint32_t box_cols, uint32_t box_rows) {
    const CUtensorMapDataType dt = m.bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == LAYER_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    cuuint64_t dims[2] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows};
    cuuint64_t strides[1] = {(cuuint64_t)m.ld * m.bytes};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = g_encode(out, dt, 2, const_cast<void*>(m.p), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_TMAP;
}

// The tensor map of a 16-bit output: its whole 16-byte pieces (store_tail).  Of a matrix
// without one it is never used.
int encode_out(CUtensorMap* out, Mat m, int dtype, uint32_t box_rows) {
    if (m.cols >= 8) m.cols &= ~7ll;
    return encode_mat(out, m, dtype, 64, box_rows);
}

template <typename... P, typename... A>
int launch_pdl(void (*kern)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3(threads, 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&lc, kern, std::forward<A>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// ---- one matrix product with its epilogue ------------------------------------------

// The operands as stored: a is [M, K] (NN, NT) or [K, M] (TN), b [K, N] (NN, TN)
// or [N, K] (NT).  A second pair continues K (b2 of kEpiGate: the second weight).
struct Product {
    Mat a, b, a2{nullptr, 0, 0, 0, 2}, b2{nullptr, 0, 0, 0, 2};
    Mat out[3] = {};
    int outs = 1;
    Mat in[2] = {};
    int ins = 0;
    long long M, N, K;
    // the kernel before this one on the stream is this call's own (and so began when everything
    // before it was complete), and it does not write b
    bool after_own = false;
    LayerParams p{};
};

// CTA pairs: 256 x 256 tiles (kEpiGate 256 x 128 of h), and for the store
// epilogue a split along K over clusters of 2 to 4 pairs.
struct PairPlan {
    int tiles, pairs, split, k_steps;
};

// Cycles a product is expected to take, to choose between the kernels and their
// splits.  A pair takes about 545 a 64-deep step of a tile, 8,500 around the steps
// and 8,500 more to exchange partials; HBM gives 3,300 bytes a cycle.  (Over 66
// products of 1 to 1024 tokens with K, N from 1024 to 14336, the choice by these two
// estimates cost 0.1 % on average and 3 % at worst against the better of the two.)
long long product_bytes(const Product& q, int weights) {
    return 2 * (weights * q.K * q.N + q.M * (q.K + q.N));
}

long long pair_cycles(const PairPlan& g, const Product& q, int weights) {
    const int waves = g.split > 1 ? 1 : ceil_div(g.tiles, g.pairs);
    const long long steps = 8500 + (long long)waves * ceil_div(g.k_steps, g.split) * 545 + (g.split > 1 ? 8500 : 0);
    const long long bytes = 9500 + product_bytes(q, weights) / 3300;
    return steps > bytes ? steps : bytes;
}

PairPlan pair_plan(const Product& q, int epi, const Ctx& c) {
    PairPlan g{};
    g.k_steps = ceil_div(q.K, 64) * (q.a2.p ? 2 : 1);
    const long long tiles = (long long)ceil_div(q.M, 256) * ceil_div(q.N, epi == kEpiGate ? 128 : 256);
    g.tiles = tiles > INT_MAX - 1024 ? INT_MAX : (int)tiles;
    g.pairs = max_pairs_of(*c.dev);
    g.split = 1;
    if (epi != kEpiStore) return g;
    PairPlan best = g;
    for (int s = 2; s <= kLayerMaxSplit; ++s) {
        g.split = s;
        if (g.k_steps / s < 4 || g.tiles > max_clusters_of(*c.dev, 2 * s)) break;
        if (pair_cycles(g, q, 1) < pair_cycles(best, q, 1)) best = g;
    }
    return best;
}

template <int LAY, int EPI, int DT, bool SPLIT>
int run_product_pair(const Product& q, const PairPlan& g, const Ctx& c) {
    using L = LayerPairLayout<EPI, SPLIT>;
    constexpr bool kAMN = LAY == kTN, kBMN = LAY != kNT;
    constexpr int dtype = DT == kBF16 ? LAYER_BF16 : LAYER_F16;
    LayerMaps tm;
    std::memset(&tm, 0, sizeof(tm));
    const Mat as[2] = {q.a, q.a2.p ? q.a2 : q.a}, bs[2] = {q.b, q.b2.p ? q.b2 : q.b};
    int rc = GEMM_OK;
    for (int i = 0; i < 2 && rc == GEMM_OK; ++i) {
        if (i == 1 && !q.a2.p && !q.b2.p) {
            tm.a[1] = tm.a[0];
            tm.b[1] = tm.b[0];
            break;
        }
        rc = encode_mat(&tm.a[i], as[i], dtype, 64, kAMN ? 64 : 128);
        if (rc == GEMM_OK) rc = encode_mat(&tm.b[i], bs[i], dtype, 64, kBMN ? 64 : kTileN / 2);
    }
    for (int i = 0; i < q.outs && rc == GEMM_OK && EPI != kEpiLossStats && EPI != kEpiLossStatsLong; ++i)
        rc = EPI == kEpiStore || EPI == kEpiGate ? encode_out(&tm.out[i], q.out[i], dtype, 32)
                                                 : encode_mat(&tm.out[i], q.out[i], dtype, 128 / q.out[i].bytes, 32);
    for (int i = 0; i < q.ins && rc == GEMM_OK; ++i) rc = encode_mat(&tm.in[i], q.in[i], dtype, 128 / q.in[i].bytes, 32);
    if (rc != GEMM_OK) return rc;

    LayerParams p = q.p;
    p.M = (int)q.M;
    p.N = (int)q.N;
    p.tiles_m = ceil_div(q.M, 256);
    p.tiles_n = ceil_div(q.N, L::kOutN);
    if ((long long)p.tiles_m * p.tiles_n > INT_MAX - 1024) return GEMM_ERR_DIM;
    p.k_switch = ceil_div(q.K, 64);
    p.k_steps = q.a2.p ? 2 * p.k_switch : p.k_switch;
    p.raster_group = 8;
    p.wait_limit = c.wait_limit;
    p.inject = c.inject;
    p.split = g.split;
    for (int i = 0; i < q.outs; ++i) {
        p.tail_out[i] = const_cast<void*>(q.out[i].p);
        p.tail_ld[i] = q.out[i].ld;
    }
    auto kern = layer_pair_kernel<LAY, EPI, DT, SPLIT>;
    static std::atomic<bool> ready[kMaxDevices];
    rc = ensure_smem_limit(kern, L::kSmem, ready[c.ordinal]);
    if (rc != GEMM_OK) return rc;
    const int clusters = SPLIT || g.tiles < g.pairs ? g.tiles : g.pairs;
    return launch_pdl(kern, dim3(2 * g.split * clusters), L::kThreads, L::kSmem, 2 * g.split, c.stream, tm, p);
}

constexpr int kSkinnyTwoSmem = 115712;  // two such CTAs fill an SM's 228 KiB
// A CTA that pushes partials holds Tensor Memory while it waits for its cluster to start, as
// the GEMM's clusters do.  Beside one of those that takes all 512 columns (and, with few
// stages configured, no more than smem_request's half of an SM's shared memory) on another
// stream, each could hold what the other's peer waits for: so no SM takes both.  (1 KiB a
// CTA is the system's.  The other forms here give Tensor Memory back before they wait.)
static_assert(kSkinnyTwoSmem + 1024 + (233472 / 2 + 1) + 1024 > 233472, "a pushing CTA beside a 512-column one");

// How the kernel for few tokens runs a product: tokens a tile, split along K,
// shared memory.
struct SkinnyPlan {
    int nt, t_tiles, tiles, split, slots, stage_bytes, smem, tmem_cols, waves, k_steps;
    int push, recv_bytes, accs;
    bool too_long;  // a run of the loss's logits would be longer than allowed
};

// As pair_cycles.  An SM takes in about 58 bytes a cycle of operands that hit L2; 8,000
// cycles around the steps, 45 a token of the tile for its way through shared memory.
long long skinny_cycles(const SkinnyPlan& g, const Product& q, int weights) {
    const long long steps = 8000 + (long long)g.waves * ceil_div(g.k_steps, g.split) * (g.stage_bytes / 58) +
                            45ll * g.nt * weights;
    const long long bytes = 6500 + product_bytes(q, weights) / 3300;
    return steps > bytes ? steps : bytes;
}

// promote: K steps of the loss's logits that may go into one accumulator.
SkinnyPlan skinny_plan(const Product& q, int epi, int sms, const int* held, int promote) {
    const bool gate = epi == kEpiGate;
    SkinnyPlan g{};
    const int most = gate ? 128 : 256;  // the fp32 partials of a tile have to fit the ring
    g.t_tiles = ceil_div(q.M, most);
    g.nt = (ceil_div(q.M, g.t_tiles) + 15) / 16 * 16;
    g.tiles = ceil_div(q.N, 128) * g.t_tiles;
    const int weights = gate ? 2 : 1, k_steps = ceil_div(q.K, 64) * (q.a2.p ? 2 : 1);
    g.stage_bytes = weights * kSkinnyTileBytes + g.nt * 128;
    const int cols = weights * g.nt;
    g.tmem_cols = cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
    // Two CTAs an SM where their accumulators are small and the ring still holds some
    // 80 KB of weights (64 KB of a gated tile's).  An SM takes in about 64 GB/s of weights
    // missing L2, so HBM's rate needs four SMs in five busy: one CTA on each, or two of a
    // gated tile's shallow rings.  The split is the least that gives so many CTAs, among
    // those whose clusters all fit at once, at two K steps each at least (one token,
    // K = N = 4096: 1, 2, 4, 6 and 8 CTAs a tile 20.4, 11.9, 8.5, 8.9 and 8.9 us; 8 tokens,
    // K = 32768, N = 1024: 8, 12 and 16 CTAs a tile 20.8, 15.9 and 14.9 us; the gated
    // block of 4096 x 14336: 2, 3 and 4 CTAs a gate and up tile 57, 65 and 61 us in all, the
    // last two in two waves).
    const int fixed = 1024 + 8 * (2 * kSkinnySlots + 2) + 16;
    const int in_flight = (kSkinnyTwoSmem - fixed) / g.stage_bytes * weights * kSkinnyTileBytes;
    const bool two = cols <= 128 && in_flight >= (gate ? 65536 : 81920);
    // (After this call's own kernel the weights' first loads run under that kernel's
    // end, and twice the CTAs start more of them: worth it where 16 steps each remain.
    // Gated block for one token, 4096 x 14336: 61.7 -> 57.0 us.  Not for the loss's logits:
    // both passes take the same plan, so that they sum them alike.)
    const int each = sms * 4 / 5;
    const bool twice = two && (gate || (q.after_own && epi != kEpiLossGrad && (long long)k_steps * g.tiles >= 32ll * each));
    const int want = twice ? 2 * each : each;
    int split = 1;
    for (int s = 2; s <= kSkinnySplit && s * 2 <= k_steps && g.tiles * split < want; ++s)
        if (g.tiles <= held[s] * (two ? 2 : 1)) split = s;
    g.split = split;
    // the loss's logits in accumulators of `promote` steps each, if Tensor Memory holds so many
    g.accs = 1;
    if (epi == kEpiLossStats || epi == kEpiLossGrad) {
        const int room = (two ? 256 : 512) / g.nt, steps = ceil_div(k_steps, split);
        g.accs = ceil_div(steps, promote);
        if (g.accs > room) {
            g.accs = room;
            g.too_long = true;
        }
        while (g.tmem_cols < g.accs * g.nt) g.tmem_cols *= 2;
    }
    // Partials of few tokens are pushed within small clusters (pulled and pushed, medians
    // of seven: one token, K = N = 4096 8.71 and 8.47 us, K = 2048, N = 8192 8.72 and 8.46;
    // four tokens 8.74 and 8.66, 8.74 and 8.49).  In larger clusters, for more tokens and
    // for two weights pulling is faster (one token, K = N = 1024, eight CTAs 3.71 and
    // 3.77; 16 tokens, K = N = 4096 8.88 and 9.04; gated block of 512 x 2048, 8 tokens, 8.51
    // and 9.30).
    const int budget = (two ? kSkinnyTwoSmem : kSmemLimit) - fixed;
    g.push = epi == kEpiStore && q.M <= kPushTokens && split > 1 && split <= kPushSplit;
    g.recv_bytes = g.push ? ceil_div(q.M, split) * split * 512 : 0;
    g.slots = (budget - g.recv_bytes) / g.stage_bytes;
    if (g.slots > kSkinnySlots) g.slots = kSkinnySlots;
    g.smem = g.slots * g.stage_bytes + g.recv_bytes + fixed;
    const int floor_smem = two ? 78848 : 118784;  // never three CTAs an SM, or two
    if (g.smem < floor_smem) g.smem = floor_smem;
    if (g.push) g.smem = kSkinnyTwoSmem;  // above
    g.waves = ceil_div((long long)g.tiles * g.split, sms);
    g.k_steps = k_steps;
    return g;
}

// [s]: how many clusters of s CTAs, one CTA an SM, the device holds at once (a
// cluster's CTAs share a GPC, so not every size packs the SMs).  Asked once per
// device and kernel.  cudaOccupancyMaxActiveClusters gives the same numbers for CTAs
// that fit an SM twice; twice as many of them run at once all the same.
template <bool WMN, int EPI, int DT>
const int* skinny_clusters(const Ctx& c) {
    static int held[kMaxDevices][kSkinnySplit + 1];
    static std::atomic<bool> known[kMaxDevices];
    if (known[c.ordinal].load(std::memory_order_acquire)) return held[c.ordinal];
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (known[c.ordinal].load(std::memory_order_relaxed)) return held[c.ordinal];
    auto kern = layer_skinny_kernel<WMN, EPI, DT, false>;
    bool can = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) == cudaSuccess;
    for (int s = 1; s <= kSkinnySplit; ++s) {
        if (s == kMaxSplit + 1)
            can = can && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3(s * 64, 1, 1);
        lc.blockDim = dim3(kThreads, 1, 1);
        lc.dynamicSmemBytes = kSmemLimit;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = s;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        int n = 0;
        held[c.ordinal][s] = can && cudaOccupancyMaxActiveClusters(&n, kern, &lc) == cudaSuccess ? n : 0;
    }
    cudaGetLastError();
    known[c.ordinal].store(true, std::memory_order_release);
    return held[c.ordinal];
}

template <bool WMN, int EPI, int DT>
int run_product_skinny(const Product& q, const SkinnyPlan& g, const Ctx& c) {
    constexpr int dtype = DT == kBF16 ? LAYER_BF16 : LAYER_F16;
    SkinnyMaps tm;
    std::memset(&tm, 0, sizeof(tm));
    SkinnyParams p;
    std::memset(&p, 0, sizeof(p));
    p.T = (int)q.M;
    p.N = (int)q.N;
    p.nt = g.nt;
    p.t_tiles = g.t_tiles;
    int rc = encode_mat(&tm.w[0], q.b, dtype, 64, WMN ? 64 : 128);
    if (rc == GEMM_OK) rc = encode_mat(&tm.x[0], q.a, dtype, 64, g.nt);
    if (rc == GEMM_OK && q.b2.p) rc = encode_mat(&tm.w[1], q.b2, dtype, 64, WMN ? 64 : 128);
    if (rc == GEMM_OK && q.a2.p) rc = encode_mat(&tm.x[1], q.a2, dtype, 64, g.nt);
    if (rc != GEMM_OK) return rc;
    p.k_switch = ceil_div(q.K, 64);
    p.k_steps = q.a2.p ? 2 * p.k_switch : p.k_switch;
    p.split = g.split;
    p.weights_early = q.after_own;
    p.slots = g.slots;
    p.stage_bytes = g.stage_bytes;
    p.accs = g.accs;
    p.recv_bytes = g.recv_bytes;
    p.tmem_cols = g.tmem_cols;
    if ((long long)g.tiles * g.split > INT_MAX) return GEMM_ERR_DIM;
    p.act = q.p.act;
    p.bias = q.p.bias;
    p.alpha = q.p.alpha;
    p.alpha_rows = q.p.alpha_rows;
    if (EPI == kEpiGateGrad) {
        p.gate = q.in[0].p;
        p.ld_gate = q.in[0].ld;
        p.up = q.in[1].p;
        p.ld_up = q.in[1].ld;
    } else if (q.ins > 0) {
        p.addend = q.in[0].p;
        p.ld_addend = q.in[0].ld;
        p.addend_f32 = q.in[0].bytes == 4;
    }
    p.out = const_cast<void*>(q.out[0].p);
    p.ld_out = q.out[0].ld;
    p.out_f32 = q.out[0].bytes == 4;
    p.keep0 = const_cast<void*>(q.out[1].p);  // (kEpiGateGrad does not read it)
    p.ld_keep0 = q.out[1].ld;
    const Mat& second = q.out[EPI == kEpiGateGrad ? 1 : 2];
    p.keep1 = const_cast<void*>(second.p);
    p.ld_keep1 = second.ld;
    p.stats = q.p.stats;
    p.target_logit = q.p.target_logit;
    p.target = q.p.target;
    p.col0 = q.p.col0;
    p.lse = q.p.lse;
    p.row_scale = q.p.row_scale;
    p.row_scale2 = q.p.row_scale2;
    p.wait_limit = c.wait_limit;
    p.inject = c.inject;
    const int smem = g.smem, split = g.split, tiles = g.tiles;
    auto start = [&](auto kern, std::atomic<bool>& ready) {
        const int r = ensure_smem_limit(kern, kSmemLimit, ready);
        return r != GEMM_OK ? r : launch_pdl(kern, dim3(tiles * split), kThreads, smem, split, c.stream, tm, p);
    };
    static std::atomic<bool> ready[2][kMaxDevices];
    if constexpr (EPI == kEpiStore)
        if (g.push) return start(layer_skinny_kernel<WMN, EPI, DT, true>, ready[1][c.ordinal]);
    return start(layer_skinny_kernel<WMN, EPI, DT, false>, ready[0][c.ordinal]);
}

// The kernel whose expected time is less; beyond kFewTokens always the pairs'.
constexpr long long kFewTokens = 1024;

template <int LAY, int EPI, int DT>
int run_product_as(const Product& q, const Ctx& c) {
    const PairPlan g = pair_plan(q, EPI, c);
    if constexpr (LAY != kTN) {
        constexpr int epi = EPI == kEpiStoreF32 ? kEpiStore : EPI;  // the output's type is a parameter there
        if (q.M <= kFewTokens) {
            const SkinnyPlan f = skinny_plan(q, EPI, c.dev->sms, skinny_clusters<LAY == kNN, epi, DT>(c), kPromote<DT>);
            constexpr int weights = EPI == kEpiGate ? 2 : 1;
            if (!f.too_long && skinny_cycles(f, q, weights) <= pair_cycles(g, q, weights))
                return run_product_skinny<LAY == kNN, epi, DT>(q, f, c);
        }
    }
    if constexpr (EPI == kEpiLossStats)
        if (g.k_steps > kPromote<DT>) return run_product_pair<LAY, kEpiLossStatsLong, DT, false>(q, g, c);
    if constexpr (EPI == kEpiLossGrad)
        if (g.k_steps > kPromote<DT>) return run_product_pair<LAY, kEpiLossGradLong, DT, false>(q, g, c);
    if constexpr (EPI == kEpiStore)
        if (g.split > 1) return run_product_pair<LAY, EPI, DT, true>(q, g, c);
    return run_product_pair<LAY, EPI, DT, false>(q, g, c);
}

template <int LAY, int EPI>
int run_product(const Product& q, int dtype, const Ctx& c) {
    return dtype == LAYER_BF16 ? run_product_as<LAY, EPI, kBF16>(q, c) : run_product_as<LAY, EPI, kF16>(q, c);
}

// ---- several products of a backward pass together -----------------------------------------

struct GradProduct {
    Product q;
    int layout;
};

template <int DT>
int run_grads_as(const GradProduct* list, int n, int longs, const Ctx& c) {
    constexpr int dtype = DT == kBF16 ? LAYER_BF16 : LAYER_F16;
    using L = LayerPairLayout<kEpiStore, false>;
    GradsMaps tm;
    std::memset(&tm, 0, sizeof(tm));
    GradsParams p;
    std::memset(&p, 0, sizeof(p));
    int rc = GEMM_OK;
    for (int i = 0; i < n && rc == GEMM_OK; ++i) {
        const Product& q = list[i].q;
        GradsProblem& g = p.q[i];
        g.a_mn = list[i].layout == kTN;
        g.b_mn = list[i].layout != kNT;
        g.M = (int)q.M;
        g.N = (int)q.N;
        g.alpha = q.p.alpha;
        g.alpha_rows = q.p.alpha_rows;
        g.tiles_m = ceil_div(q.M, 256);
        g.tiles_n = ceil_div(q.N, 256);
        g.k_switch = ceil_div(q.K, 64);
        g.k_steps = q.a2.p ? 2 * g.k_switch : g.k_switch;
        rc = encode_mat(&tm.a[i], q.a, dtype, 64, g.a_mn ? 64 : 128);
        if (rc == GEMM_OK) rc = encode_mat(&tm.b[i], q.b, dtype, 64, g.b_mn ? 64 : 128);
        if (rc == GEMM_OK && q.a2.p) {
            rc = encode_mat(&tm.a[kGradsProblems], q.a2, dtype, 64, g.a_mn ? 64 : 128);
            if (rc == GEMM_OK) rc = encode_mat(&tm.b[kGradsProblems], q.b2, dtype, 64, g.b_mn ? 64 : 128);
        }
        if (rc == GEMM_OK) rc = encode_out(&tm.out[i], q.out[0], dtype, 32);
        g.out = const_cast<void*>(q.out[0].p);
        g.ld_out = q.out[0].ld;
    }
    if (rc != GEMM_OK) return rc;
    p.longs = longs;
    for (int i = 0; i < n; ++i) p.tiles[i < p.longs ? 0 : 1] += p.q[i].tiles_m * p.q[i].tiles_n;
    const int pairs = max_pairs_of(*c.dev);
    p.rounds = p.tiles[0] / pairs;
    p.rem = p.tiles[0] % pairs;
    if (p.rem > 0) {
        const int shorter = p.q[longs].k_steps;
        p.d = (p.q[0].k_steps + shorter / 2) / shorter;
        const int most = p.tiles[1] / (pairs - p.rem);
        if (p.d > most) p.d = most;
    }
    p.raster_group = 8;
    p.wait_limit = c.wait_limit;
    p.inject = c.inject;
    auto kern = layer_grads_kernel<DT>;
    static std::atomic<bool> ready[kMaxDevices];
    rc = ensure_smem_limit(kern, L::kSmem, ready[c.ordinal]);
    if (rc != GEMM_OK) return rc;
    return launch_pdl(kern, dim3(2 * pairs), kThreads, L::kSmem, 2, c.stream, tm, p);
}

// Cycles of one product by itself, and of a tile of it among others; the estimates
// above, with at least 6,000 cycles a tile for writing it: a weight gradient over few
// tokens is all writing.
long long alone_cycles(const GradProduct& p, const Ctx& c) {
    const Product& q = p.q;
    const PairPlan g = pair_plan(q, kEpiStore, c);
    const long long tile = ceil_div(g.k_steps, g.split) * 545ll;
    long long cost = 8500 + (g.split > 1 ? 8500 : 0) + (g.split > 1 ? 1 : ceil_div(g.tiles, g.pairs)) * (tile > 6000 ? tile : 6000);
    const long long bytes = 9500 + product_bytes(q, 1) / 3300;
    if (cost < bytes) cost = bytes;
    if (p.layout != kTN && q.M <= kFewTokens) {
        const long long few = skinny_cycles(skinny_plan(q, kEpiStore, c.dev->sms, skinny_clusters<false, kEpiStore, kF16>(c), 0), q, 1);
        if (few < cost) cost = few;
    }
    return cost;
}

long long together_cycles(const GradProduct* list, int n, const Ctx& c) {
    long long cycles = 0, longest = 0, tiles = 0;
    for (int i = 0; i < n; ++i) {
        const Product& q = list[i].q;
        const long long here = (long long)ceil_div(q.M, 256) * ceil_div(q.N, 256);
        const long long steps = ceil_div(q.K, 64) * (q.a2.p ? 2ll : 1ll) * 545, tile = steps > 6000 ? steps : 6000;
        tiles += here;
        cycles += here * tile;
        if (longest < tile) longest = tile;
    }
    if (tiles > INT_MAX / 2) return LLONG_MAX / 2;
    const int pairs = max_pairs_of(*c.dev);
    const long long spread = (cycles + pairs - 1) / pairs;
    return 8500 + (spread > longest ? spread : longest);
}

int run_alone(const GradProduct& g, int dtype, const Ctx& c) {
    switch (g.layout) {
        case kNN: return run_product<kNN, kEpiStore>(g.q, dtype, c);
        case kNT: return run_product<kNT, kEpiStore>(g.q, dtype, c);
        default: return run_product<kTN, kEpiStore>(g.q, dtype, c);
    }
}

int run_together(GradProduct* list, int n, int dtype, const Ctx& c) {
    if (n == 1) return run_alone(list[0], dtype, c);
    // the group of the larger K goes first
    int longs = 1;
    if (list[0].q.K * (list[0].q.a2.p ? 2 : 1) < list[1].q.K) {
        std::rotate(list, list + 1, list + n);
        longs = n - 1;
    }
    return dtype == LAYER_BF16 ? run_grads_as<kBF16>(list, n, longs, c) : run_grads_as<kF16>(list, n, longs, c);
}

// Products with the plain store epilogue, of which list[0] has its own K and the
// others share theirs: one after the other, all together, or list[0] alone and the
// others together, whichever is expected to take least.  (Over 54 backward passes of 8
// to 4096 tokens, widths 512 to 14336, the choice between the first two cost 0.4 % on
// average; the third: gated block of 8 tokens, 512 x 2048, 25.5 together, 15.3 so.)
int run_grads(GradProduct* list, int n, int dtype, const Ctx& c) {
    if (n <= 1) return n == 1 ? run_alone(list[0], dtype, c) : GEMM_OK;
    long long apart = 0;
    for (int i = 0; i < n; ++i) apart += alone_cycles(list[i], c);
    const long long together = together_cycles(list, n, c);
    const long long rest = n > 2 ? alone_cycles(list[0], c) + together_cycles(list + 1, n - 1, c) : LLONG_MAX;
    if (together <= apart && together <= rest) return run_together(list, n, dtype, c);
    int rc = run_alone(list[0], dtype, c);
    if (rc == GEMM_OK && rest <= apart) return run_together(list + 1, n - 1, dtype, c);
    for (int i = 1; i < n && rc == GEMM_OK; ++i) rc = run_alone(list[i], dtype, c);
    return rc;
}

// A weight gradient over no tokens is zero.
int zero_mat(const Mat& m, const Ctx& c) {
    if (!m.p || empty(m)) return GEMM_OK;
    if (cudaMemset2DAsync(const_cast<void*>(m.p), (size_t)m.ld * m.bytes, 0, (size_t)m.cols * m.bytes, (size_t)m.rows,
                          c.stream) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

int check_all(std::initializer_list<Mat> mats) {
    for (const Mat& m : mats) {
        const int rc = check_mat(m);
        if (rc != GEMM_OK) return rc;
    }
    return GEMM_OK;
}

// ---- linear layer ---------------------------------------------------------------------

int check_workspace(const void* ws, long long have, size_t need) {
    if (need == 0) return GEMM_OK;
    if (!ws) return GEMM_ERR_NULL;
    if ((uintptr_t)ws & 255) return GEMM_ERR_ALIGN;
    if (have < 0 || (size_t)have < need) return GEMM_ERR_WORKSPACE;
    return GEMM_OK;
}

struct LinearGradPlan {
    bool slope;     // dpre is a matrix of its own
    bool sums;      // dbias
    int row_blocks;
    size_t dpre_at, partial_at, bytes;
};

LinearGradPlan linear_grad_plan(const linear_grad_args& a) {
    LinearGradPlan g{};
    g.slope = a.act != LAYER_ACT_NONE && (a.dx || a.dw);
    g.sums = a.dbias != nullptr;
    g.row_blocks = ceil_div(a.tokens, kSlopeRows);
    g.partial_at = g.slope ? align256((size_t)a.tokens * pad8(a.n) * 2) : 0;
    g.bytes = g.partial_at + (g.sums ? align256((size_t)g.row_blocks * a.n * 4) : 0);
    return g;
}

template <int DT>
int run_slope(const SlopeParams& sp, void* dbias, int row_blocks, const Ctx& c) {
    int rc = launch_pdl(layer_slope_kernel<DT>, dim3(sp.col_blocks * row_blocks), 256, 0, 1, c.stream, sp);
    if (rc == GEMM_OK && dbias)
        rc = launch_pdl(layer_column_sum_kernel<DT>, dim3(ceil_div(sp.cols, 32)), 256, 0, 1, c.stream,
                        (const float*)sp.partial, dbias, row_blocks, sp.cols);
    return rc;
}

// ---- vocabulary cross entropy ------------------------------------------------------------

constexpr int kLossPart = 128;  // vocabulary columns per part of the statistics

struct LossPlan {
    int parts;
    size_t target_at, row_loss_at, bytes;
};

LossPlan loss_plan(const loss_args& a) {
    LossPlan g{};
    g.parts = ceil_div(a.vocab, kLossPart);
    g.target_at = align256((size_t)g.parts * a.tokens * sizeof(float2));
    g.row_loss_at = g.target_at + align256((size_t)a.tokens * 4);
    g.bytes = g.row_loss_at + align256((size_t)a.tokens * 4);
    return g;
}

// Backward: weights and the unscale factor, d of one piece, dh's running sum.  With
// by_rows dh's d is scaled row by row (layer_loss_weights_kernel): two more vectors, and a
// d of its own where dw is wanted too.
struct LossGradPlan {
    long long piece;
    bool by_rows;
    int copies;
    size_t unscale_at, row_weight_at, row_unscale_at, d_at, d2_at, sum_at, bytes;
};

LossGradPlan loss_grad_plan(const loss_grad_args& a, long long piece) {
    LossGradPlan g{};
    g.piece = piece < a.vocab ? piece : a.vocab;
    g.unscale_at = align256((size_t)a.tokens * 4);
    g.by_rows = a.reduction == LAYER_LOSS_NONE && a.dtype == LAYER_F16 && a.dh;
    g.copies = g.by_rows && a.dw ? 2 : 1;
    g.row_weight_at = g.unscale_at + 256;
    g.row_unscale_at = g.row_weight_at + (g.by_rows ? g.unscale_at : 0);
    g.d_at = g.row_unscale_at + (g.by_rows ? g.unscale_at : 0);
    const size_t d_bytes = align256((size_t)a.tokens * pad8(g.piece) * 2);
    g.d2_at = g.d_at + (g.copies - 1) * d_bytes;
    g.sum_at = g.d2_at + d_bytes;
    g.bytes = g.sum_at + (g.piece < a.vocab && a.dh ? align256((size_t)a.tokens * ((a.dim + 3) & ~3ll) * 4) : 0);
    return g;
}

int check_loss_grad(const loss_grad_args& a) {
    const int rc = check_dtype_act(a.dtype, 0);
    if (rc != GEMM_OK) return rc;
    if (a.reduction < LAYER_LOSS_NONE || a.reduction > LAYER_LOSS_SUM) return GEMM_ERR_CONFIG;
    if (!dims_ok({a.dim, a.vocab}, a.tokens)) return GEMM_ERR_DIM;
    return GEMM_OK;
}

// ---- gradient clipping -----------------------------------------------------------------------

constexpr int kClipBig = 1000;     // tensors a launch takes; the small table travels faster
constexpr int kClipSmall = 48;
constexpr int kClipBlocksPerSm = 8;
constexpr int kClipMaxBlocks = 256 * kClipBlocksPerSm;  // partial sums per launch

template <int CAP>
int run_clip(const grad_clip_args& a, long long entries, const Ctx& c) {
    float* partial = static_cast<float*>(a.workspace);
    static_assert(sizeof(ClipTable<kClipBig>) < 32000, "kernel parameters");
    const int max_blocks = c.dev->sms * kClipBlocksPerSm < kClipMaxBlocks ? c.dev->sms * kClipBlocksPerSm : kClipMaxBlocks;
    int parts = 0;
    ClipTable<CAP> t;
    t.chunk = kClipMostChunk;
    while (t.chunk > kClipLeastChunk && entries / t.chunk < 4ll * c.dev->sms) t.chunk /= 2;
    // both passes cut the tensors into the same tables, so `parts` ends alike
    for (int pass = 0; pass < 2; ++pass) {
        const int all_parts = parts;
        long long i = 0;
        int launches = 0;
        while (i < a.tensors || (launches == 0)) {
            t.tensors = 0;
            t.chunks = 0;
            while (i < a.tensors && t.tensors < CAP) {
                const long long n = a.count[i];
                if (n > 0) {
                    const long long ch = (n + t.chunk - 1) / t.chunk;
                    if (t.chunks + ch > INT_MAX / 2) {
                        if (t.tensors == 0) return GEMM_ERR_DIM;
                        break;
                    }
                    t.first[t.tensors] = t.chunks;
                    t.e[t.tensors] = ClipEntry{a.src[i], a.dst[i], n * 4 + a.dtype[i]};
                    t.chunks += (int)ch;
                    ++t.tensors;
                }
                ++i;
            }
            ++launches;
            const int blocks = t.chunks < 1 ? 1 : t.chunks < max_blocks ? t.chunks : max_blocks;
            int rc;
            if (pass == 0) {
                rc = launch_pdl(clip_norm_kernel<CAP>, dim3(blocks), kClipThreads, 0, 1, c.stream, t, partial + parts);
                parts += blocks;
            } else {
                rc = launch_pdl(clip_scale_kernel<CAP>, dim3(blocks), kClipThreads, 0, 1, c.stream, t,
                                (const float*)partial, all_parts, (float)a.max_norm, (float)a.eps, launches == 1 ? a.norm : nullptr);
            }
            if (rc != GEMM_OK) return rc;
        }
    }
    return GEMM_OK;
}

}  // namespace

extern "C" {

int linear_forward(const linear_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const linear_args& a = *args;
    int rc = check_dtype_act(a.dtype, a.act);
    if (rc != GEMM_OK) return rc;
    if (!dims_ok({a.k, a.n}, a.tokens)) return GEMM_ERR_DIM;
    if (a.tokens == 0) return GEMM_OK;
    const Mat x = mat16(a.x, a.tokens, a.k, a.ldx), w = mat16(a.w, a.k, a.n, a.ldw);
    const Mat y = mat16(a.y, a.tokens, a.n, a.ldy);
    const Mat r = mat16(a.residual, a.tokens, a.n, a.ldr), pre = mat16(a.preact, a.tokens, a.n, a.ldp);
    if ((rc = check_all({x, w, y})) != GEMM_OK) return rc;
    if (r.p && (rc = check_mat(r)) != GEMM_OK) return rc;
    if (pre.p && (rc = check_mat(pre)) != GEMM_OK) return rc;
    if ((uintptr_t)a.bias & 1) return GEMM_ERR_ALIGN;
    const bool in_place = r.p == y.p && a.ldr == a.ldy;
    const Span wr[] = {span_of(y), span_of(pre)};
    const Span rd[] = {span_of(x), span_of(w), span_of(a.bias, (uint64_t)a.n * 2), in_place ? Span{0, 0} : span_of(r)};
    if (overlaps(wr, 2, rd, 4)) return GEMM_ERR_ALIAS;
    if (in_place && r.p) {
        const Span p2[] = {span_of(pre)}, r2[] = {span_of(r)};
        if (overlaps(p2, 1, r2, 1)) return GEMM_ERR_ALIAS;
    }
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    Product q;
    q.a = x;
    q.b = w;
    q.M = a.tokens;
    q.N = a.n;
    q.K = a.k;
    q.out[0] = y;
    if (pre.p) {
        q.out[1] = pre;
        q.outs = 2;
        q.p.keep = 1;
    }
    if (r.p) {
        q.in[0] = r;
        q.ins = 1;
        q.p.addend = 1;
    }
    q.p.bias = a.bias;
    q.p.act = (int)a.act;
    return run_product<kNN, kEpiStore>(q, (int)a.dtype, c);
}

int linear_backward_workspace(const linear_grad_args* args, size_t* bytes) {
    if (!args || !bytes) return GEMM_ERR_NULL;
    const int rc = check_dtype_act(args->dtype, args->act);
    if (rc != GEMM_OK) return rc;
    if (!dims_ok({args->k, args->n}, args->tokens)) return GEMM_ERR_DIM;
    *bytes = linear_grad_plan(*args).bytes;
    return GEMM_OK;
}

int linear_backward(const linear_grad_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const linear_grad_args& a = *args;
    int rc = check_dtype_act(a.dtype, a.act);
    if (rc != GEMM_OK) return rc;
    if (!dims_ok({a.k, a.n}, a.tokens)) return GEMM_ERR_DIM;
    const Mat dy = mat16(a.dy, a.tokens, a.n, a.lddy), x = mat16(a.x, a.tokens, a.k, a.ldx);
    const Mat w = mat16(a.w, a.k, a.n, a.ldw), pre = mat16(a.preact, a.tokens, a.n, a.ldp);
    const Mat dx = mat16(a.dx, a.tokens, a.k, a.lddx), dw = mat16(a.dw, a.k, a.n, a.lddw);
    if ((rc = check_mat(dy)) != GEMM_OK) return rc;
    if (a.act != LAYER_ACT_NONE && (rc = check_mat(pre)) != GEMM_OK) return rc;
    if (a.dx && ((rc = check_all({w, dx})) != GEMM_OK)) return rc;
    if (a.dw && ((rc = check_all({x, dw})) != GEMM_OK)) return rc;
    if ((uintptr_t)a.dbias & 1) return GEMM_ERR_ALIGN;
    const LinearGradPlan g = linear_grad_plan(a);
    if ((long long)g.row_blocks * ceil_div(a.n, kSlopeCols) > INT_MAX) return GEMM_ERR_DIM;
    if (a.tokens > 0 && (rc = check_workspace(a.workspace, a.workspace_bytes, g.bytes)) != GEMM_OK) return rc;
    const Span wr[] = {span_of(dx), span_of(dw), span_of(a.dbias, (uint64_t)a.n * 2),
                       span_of(g.bytes ? a.workspace : nullptr, g.bytes)};
    const Span rd[] = {span_of(dy), a.dw ? span_of(x) : Span{0, 0}, a.dx ? span_of(w) : Span{0, 0},
                       a.act != LAYER_ACT_NONE ? span_of(pre) : Span{0, 0}};
    if (overlaps(wr, 4, rd, 4)) return GEMM_ERR_ALIAS;
    if (!a.dx && !a.dw && !a.dbias) return GEMM_OK;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    if (a.tokens == 0) {
        if ((rc = zero_mat(dw, c)) != GEMM_OK) return rc;
        return a.dbias ? zero_mat(Mat{a.dbias, 1, a.n, a.n, 2}, c) : GEMM_OK;
    }
    char* ws = static_cast<char*>(a.workspace);
    Mat dpre = dy;
    if (g.slope) dpre = mat16(ws, a.tokens, a.n, pad8(a.n));
    if (g.slope || g.sums) {
        SlopeParams sp{};
        sp.dy = a.dy;
        sp.ld_dy = a.lddy;
        sp.pre = a.act != LAYER_ACT_NONE ? a.preact : nullptr;
        sp.ld_pre = a.ldp;
        sp.dpre = g.slope ? ws : nullptr;
        sp.ld_dpre = dpre.ld;
        sp.partial = g.sums ? reinterpret_cast<float*>(ws + g.partial_at) : nullptr;
        sp.rows = (int)a.tokens;
        sp.cols = (int)a.n;
        sp.act = (int)a.act;
        sp.col_blocks = ceil_div(a.n, kSlopeCols);
        rc = a.dtype == LAYER_BF16 ? run_slope<kBF16>(sp, a.dbias, g.row_blocks, c)
                                   : run_slope<kF16>(sp, a.dbias, g.row_blocks, c);
        if (rc != GEMM_OK) return rc;
    }
    GradProduct list[2];
    int n = 0;
    if (a.dx) {
        Product& q = list[n].q;
        list[n++].layout = kNT;
        q.a = dpre;
        q.b = w;
        q.M = a.tokens;
        q.N = a.k;
        q.K = a.n;
        q.out[0] = dx;
        q.after_own = g.slope || g.sums;
    }
    if (a.dw) {
        Product& q = list[n].q;
        list[n++].layout = kTN;
        q.a = x;
        q.b = dpre;
        q.M = a.k;
        q.N = a.n;
        q.K = a.tokens;
        q.out[0] = dw;
    }
    return run_grads(list, n, (int)a.dtype, c);
}

int gated_ffn_forward(const gated_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const gated_args& a = *args;
    int rc = check_dtype_act(a.dtype, a.act);
    if (rc != GEMM_OK) return rc;
    if (!dims_ok({a.dim, a.ffn, a.dim_out}, a.tokens)) return GEMM_ERR_DIM;
    if (!a.gate != !a.up) return GEMM_ERR_NULL;
    if (a.tokens == 0) return GEMM_OK;
    const Mat x = mat16(a.x, a.tokens, a.dim, a.ldx);
    const Mat wg = mat16(a.w_gate, a.dim, a.ffn, a.ldw_gate), wu = mat16(a.w_up, a.dim, a.ffn, a.ldw_up);
    const Mat wd = mat16(a.w_down, a.ffn, a.dim_out, a.ldw_down);
    const Mat y = mat16(a.y, a.tokens, a.dim_out, a.ldy), r = mat16(a.residual, a.tokens, a.dim_out, a.ldr);
    const Mat h = mat16(a.hidden, a.tokens, a.ffn, a.ld_hidden);
    const Mat g = mat16(a.gate, a.tokens, a.ffn, a.ld_gate), u = mat16(a.up, a.tokens, a.ffn, a.ld_up);
    if ((rc = check_all({x, wg, wu, wd, y, h})) != GEMM_OK) return rc;
    if (r.p && (rc = check_mat(r)) != GEMM_OK) return rc;
    if (g.p && (rc = check_all({g, u})) != GEMM_OK) return rc;
    const bool in_place = r.p == y.p && a.ldr == a.ldy;
    const Span wr[] = {span_of(y), span_of(h), span_of(g), span_of(u)};
    const Span rd[] = {span_of(x), span_of(wg), span_of(wu), span_of(wd), in_place ? Span{0, 0} : span_of(r)};
    if (overlaps(wr, 4, rd, 5)) return GEMM_ERR_ALIAS;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    Product q;
    q.a = x;
    q.b = wg;
    q.b2 = wu;
    q.M = a.tokens;
    q.N = a.ffn;
    q.K = a.dim;
    q.out[0] = h;
    if (g.p) {
        q.out[1] = g;
        q.out[2] = u;
        q.outs = 3;
        q.p.keep = 1;
    }
    q.p.act = (int)a.act;
    if ((rc = run_product<kNN, kEpiGate>(q, (int)a.dtype, c)) != GEMM_OK) return rc;
    Product d;
    d.after_own = true;
    d.a = h;
    d.b = wd;
    d.M = a.tokens;
    d.N = a.dim_out;
    d.K = a.ffn;
    d.out[0] = y;
    if (r.p) {
        d.in[0] = r;
        d.ins = 1;
        d.p.addend = 1;
    }
    return run_product<kNN, kEpiStore>(d, (int)a.dtype, c);
}

int gated_ffn_backward_workspace(const gated_grad_args* args, size_t* bytes) {
    if (!args || !bytes) return GEMM_ERR_NULL;
    const int rc = check_dtype_act(args->dtype, args->act);
    if (rc != GEMM_OK) return rc;
    if (!dims_ok({args->dim, args->ffn, args->dim_out}, args->tokens)) return GEMM_ERR_DIM;
    *bytes = args->dx || args->dw_gate || args->dw_up ? 2 * align256((size_t)args->tokens * pad8(args->ffn) * 2) : 0;
    return GEMM_OK;
}

int gated_ffn_backward(const gated_grad_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const gated_grad_args& a = *args;
    size_t need = 0;
    int rc = gated_ffn_backward_workspace(args, &need);
    if (rc != GEMM_OK) return rc;
    if (!a.dw_gate != !a.dw_up) return GEMM_ERR_NULL;
    const long long T = a.tokens;
    const Mat dy = mat16(a.dy, T, a.dim_out, a.lddy), x = mat16(a.x, T, a.dim, a.ldx);
    const Mat wg = mat16(a.w_gate, a.dim, a.ffn, a.ldw_gate), wu = mat16(a.w_up, a.dim, a.ffn, a.ldw_up);
    const Mat wd = mat16(a.w_down, a.ffn, a.dim_out, a.ldw_down);
    const Mat gt = mat16(a.gate, T, a.ffn, a.ld_gate), up = mat16(a.up, T, a.ffn, a.ld_up);
    const Mat hid = mat16(a.hidden, T, a.ffn, a.ld_hidden);
    const Mat dx = mat16(a.dx, T, a.dim, a.lddx);
    const Mat dwg = mat16(a.dw_gate, a.dim, a.ffn, a.lddw_gate), dwu = mat16(a.dw_up, a.dim, a.ffn, a.lddw_up);
    const Mat dwd = mat16(a.dw_down, a.ffn, a.dim_out, a.lddw_down);
    const bool inner = a.dx || a.dw_gate;  // dgate and dup are needed
    if (!inner && !a.dw_down) return GEMM_OK;
    if ((rc = check_mat(dy)) != GEMM_OK) return rc;
    if (inner && (rc = check_all({wd, gt, up})) != GEMM_OK) return rc;
    if (a.dx && (rc = check_all({wg, wu, dx})) != GEMM_OK) return rc;
    if (a.dw_gate && (rc = check_all({x, dwg, dwu})) != GEMM_OK) return rc;
    if (a.dw_down && (rc = check_all({hid, dwd})) != GEMM_OK) return rc;
    if (T > 0 && (rc = check_workspace(a.workspace, a.workspace_bytes, need)) != GEMM_OK) return rc;
    const Span none{0, 0};
    const Span wr[] = {span_of(dx), span_of(dwg), span_of(dwu), span_of(dwd), span_of(need ? a.workspace : nullptr, need)};
    const Span rd[] = {span_of(dy), a.dw_gate ? span_of(x) : none, a.dx ? span_of(wg) : none, a.dx ? span_of(wu) : none,
                       inner ? span_of(wd) : none, inner ? span_of(gt) : none, inner ? span_of(up) : none,
                       a.dw_down ? span_of(hid) : none};
    if (overlaps(wr, 5, rd, 8)) return GEMM_ERR_ALIAS;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    if (T == 0) {
        for (const Mat& m : {dwg, dwu, dwd})
            if ((rc = zero_mat(m, c)) != GEMM_OK) return rc;
        return GEMM_OK;
    }
    char* ws = static_cast<char*>(a.workspace);
    const Mat dg = mat16(ws, T, a.ffn, pad8(a.ffn)), du = mat16(ws + need / 2, T, a.ffn, pad8(a.ffn));
    const int dtype = (int)a.dtype;
    if (inner) {
        Product q;
        q.a = dy;
        q.b = wd;
        q.M = T;
        q.N = a.ffn;
        q.K = a.dim_out;
        q.out[0] = dg;
        q.out[1] = du;
        q.outs = 2;
        q.in[0] = gt;
        q.in[1] = up;
        q.ins = 2;
        q.p.act = (int)a.act;
        if ((rc = run_product<kNT, kEpiGateGrad>(q, dtype, c)) != GEMM_OK) return rc;
    }
    GradProduct list[4];
    int n = 0;
    if (a.dx) {
        Product& q = list[n].q;
        list[n++].layout = kNT;
        q.after_own = true;
        q.a = dg;
        q.a2 = du;
        q.b = wg;
        q.b2 = wu;
        q.M = T;
        q.N = a.dim;
        q.K = a.ffn;
        q.out[0] = dx;
    }
    auto weight_grad = [&](const Mat& in, const Mat& d, const Mat& out) {
        Product& q = list[n].q;
        list[n++].layout = kTN;
        q.a = in;
        q.b = d;
        q.M = in.cols;
        q.N = d.cols;
        q.K = T;
        q.out[0] = out;
    };
    if (a.dw_gate) {
        weight_grad(x, dg, dwg);
        weight_grad(x, du, dwu);
    }
    if (a.dw_down) weight_grad(hid, dy, dwd);
    return run_grads(list, n, dtype, c);
}

int linear_cross_entropy_workspace(const loss_args* args, size_t* bytes) {
    if (!args || !bytes) return GEMM_ERR_NULL;
    const int rc = check_dtype_act(args->dtype, 0);
    if (rc != GEMM_OK) return rc;
    if (args->reduction < LAYER_LOSS_NONE || args->reduction > LAYER_LOSS_SUM) return GEMM_ERR_CONFIG;
    if (!dims_ok({args->dim, args->vocab}, args->tokens)) return GEMM_ERR_DIM;
    *bytes = args->tokens > 0 ? loss_plan(*args).bytes : 0;
    return GEMM_OK;
}

int linear_cross_entropy(const loss_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const loss_args& a = *args;
    size_t need = 0;
    int rc = linear_cross_entropy_workspace(args, &need);
    if (rc != GEMM_OK) return rc;
    const Mat h = mat16(a.h, a.tokens, a.dim, a.ldh), w = mat16(a.w, a.vocab, a.dim, a.ldw);
    const bool each = a.reduction == LAYER_LOSS_NONE;
    if (!a.loss && (a.tokens > 0 || !each)) return GEMM_ERR_NULL;
    if ((uintptr_t)a.loss & 3) return GEMM_ERR_ALIGN;
    if (a.tokens > 0) {
        if (!a.target || !a.lse) return GEMM_ERR_NULL;
        if (((uintptr_t)a.target & 7) || ((uintptr_t)a.lse & 3)) return GEMM_ERR_ALIGN;
        if ((rc = check_all({h, w})) != GEMM_OK) return rc;
        if ((rc = check_workspace(a.workspace, a.workspace_bytes, need)) != GEMM_OK) return rc;
        const Span wr[] = {span_of(a.loss, (uint64_t)(each ? a.tokens : 1) * 4), span_of(a.lse, (uint64_t)a.tokens * 4),
                           span_of(a.workspace, need)};
        const Span rd[] = {span_of(h), span_of(w), span_of(a.target, (uint64_t)a.tokens * 8)};
        if (overlaps(wr, 3, rd, 3)) return GEMM_ERR_ALIAS;
    }
    Ctx c;
    if (a.tokens == 0 && each) return GEMM_OK;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    if (a.tokens == 0) return zero_mat(Mat{a.loss, 1, 1, 1, 4}, c);
    const LossPlan g = loss_plan(a);
    char* ws = static_cast<char*>(a.workspace);
    Product q;
    q.a = h;
    q.b = w;
    q.M = a.tokens;
    q.N = a.vocab;
    q.K = a.dim;
    q.p.stats = reinterpret_cast<float2*>(ws);
    q.p.target_logit = reinterpret_cast<float*>(ws + g.target_at);
    q.p.target = a.target;
    if ((rc = run_product<kNT, kEpiLossStats>(q, (int)a.dtype, c)) != GEMM_OK) return rc;
    LossParams lp{};
    lp.stats = q.p.stats;
    lp.target_logit = q.p.target_logit;
    lp.target = a.target;
    lp.row_loss = each ? a.loss : reinterpret_cast<float*>(ws + g.row_loss_at);
    lp.lse = a.lse;
    lp.rows = (int)a.tokens;
    lp.parts = g.parts;
    lp.vocab = a.vocab;
    lp.ignore_index = a.ignore_index;
    if (!each && a.tokens <= 32) {
        lp.total = a.loss;
        lp.mean = a.reduction == LAYER_LOSS_MEAN;
    }
    if ((rc = launch_pdl(layer_loss_rows_kernel, dim3(ceil_div(a.tokens, 32)), 1024, 0, 1, c.stream, lp)) != GEMM_OK) return rc;
    if (each || lp.total) return GEMM_OK;
    return launch_pdl(layer_loss_sum_kernel, dim3(1), 1024, 0, 1, c.stream, (const float*)lp.row_loss, a.target, a.loss,
                      (int)a.tokens, a.ignore_index, (int)(a.reduction == LAYER_LOSS_MEAN));
}

int linear_cross_entropy_backward_workspace(const loss_grad_args* args, long long piece, size_t* bytes) {
    if (!args || !bytes) return GEMM_ERR_NULL;
    const int rc = check_loss_grad(*args);
    if (rc != GEMM_OK) return rc;
    if (piece < 256 || piece % 256 != 0) return GEMM_ERR_DIM;
    *bytes = args->tokens > 0 ? loss_grad_plan(*args, piece).bytes : 0;
    return GEMM_OK;
}

int linear_cross_entropy_backward(const loss_grad_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const loss_grad_args& a = *args;
    int rc = check_loss_grad(a);
    if (rc != GEMM_OK) return rc;
    if (!a.dh && !a.dw) return GEMM_OK;
    const long long T = a.tokens;
    const Mat h = mat16(a.h, T, a.dim, a.ldh), w = mat16(a.w, a.vocab, a.dim, a.ldw);
    const Mat dh = mat16(a.dh, T, a.dim, a.lddh), dw = mat16(a.dw, a.vocab, a.dim, a.lddw);
    if (a.dw && (rc = check_mat(dw)) != GEMM_OK) return rc;
    Ctx c;
    if (T == 0) {
        if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
        return zero_mat(dw, c);
    }
    if (a.dh && (rc = check_mat(dh)) != GEMM_OK) return rc;
    if ((rc = check_all({h, w})) != GEMM_OK) return rc;
    if (!a.target || !a.lse || !a.grad_loss) return GEMM_ERR_NULL;
    if (((uintptr_t)a.target & 7) || ((uintptr_t)a.lse & 3) || ((uintptr_t)a.grad_loss & 3)) return GEMM_ERR_ALIGN;
    // the largest piece the workspace holds: all of the vocabulary, else a multiple of 256
    if (!a.workspace) return GEMM_ERR_NULL;
    if ((uintptr_t)a.workspace & 255) return GEMM_ERR_ALIGN;
    const size_t have = a.workspace_bytes < 0 ? 0 : (size_t)a.workspace_bytes;
    long long piece = a.vocab;
    if (loss_grad_plan(a, piece).bytes > have) {
        const size_t fixed = loss_grad_plan(a, 256 < a.vocab ? 256 : a.vocab).bytes;
        if (256 >= a.vocab || fixed > have) return GEMM_ERR_WORKSPACE;
        piece = 256 + (long long)((have - fixed) / ((size_t)T * 2 * loss_grad_plan(a, 256).copies)) / 256 * 256;
        if (piece >= a.vocab) piece = (a.vocab - 1) / 256 * 256;
        while (piece > 256 && loss_grad_plan(a, piece).bytes > have) piece -= 256;
    }
    const LossGradPlan g = loss_grad_plan(a, piece);
    const Span wr[] = {span_of(dh), span_of(dw), span_of(a.workspace, g.bytes)};
    const Span rd[] = {span_of(h), span_of(w), span_of(a.target, (uint64_t)T * 8), span_of(a.lse, (uint64_t)T * 4),
                       span_of(a.grad_loss, (uint64_t)(a.reduction == LAYER_LOSS_NONE ? T : 1) * 4)};
    if (overlaps(wr, 3, rd, 5)) return GEMM_ERR_ALIAS;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    char* ws = static_cast<char*>(a.workspace);
    float* weight = reinterpret_cast<float*>(ws);
    float* unscale = reinterpret_cast<float*>(ws + g.unscale_at);
    const int dtype = (int)a.dtype;
    float* row_weight = g.by_rows ? reinterpret_cast<float*>(ws + g.row_weight_at) : nullptr;
    float* row_unscale = g.by_rows ? reinterpret_cast<float*>(ws + g.row_unscale_at) : nullptr;
    rc = launch_pdl(layer_loss_weights_kernel, dim3(1), 1024, 0, 1, c.stream, a.grad_loss, a.target, weight, unscale, row_weight,
                    row_unscale, (int)T, a.vocab, a.ignore_index, (int)a.reduction);
    if (rc != GEMM_OK) return rc;
    const long long ldsum = (a.dim + 3) & ~3ll;
    for (long long v0 = 0; v0 < a.vocab; v0 += piece) {
        const long long n = a.vocab - v0 < piece ? a.vocab - v0 : piece;
        const bool first = v0 == 0, last = v0 + n == a.vocab;
        const Mat d = mat16(ws + g.d_at, T, n, pad8(g.piece));   // dw's, or both's
        const Mat d2 = mat16(ws + g.d2_at, T, n, pad8(g.piece));  // dh's
        const Mat wp = mat16(static_cast<const char*>(a.w) + (size_t)v0 * a.ldw * 2, n, a.dim, a.ldw);
        Product q;
        q.after_own = true;
        q.a = h;
        q.b = wp;
        q.M = T;
        q.N = n;
        q.K = a.dim;
        q.out[0] = d;
        q.p.target = a.target;
        q.p.col0 = (int)v0;
        q.p.lse = a.lse;
        q.p.row_scale = g.by_rows && !a.dw ? row_weight : weight;
        if (g.copies == 2) {
            q.out[1] = d2;
            q.outs = 2;
            q.p.keep = 1;
            q.p.row_scale2 = row_weight;
        }
        if ((rc = run_product<kNT, kEpiLossGrad>(q, dtype, c)) != GEMM_OK) return rc;
        GradProduct list[2];
        int count = 0;
        if (a.dh) {
            // dh = d w, over the pieces in fp32; the last sum is unscaled and rounded
            const Mat sum = Mat{ws + g.sum_at, T, a.dim, ldsum, 4};
            Product& s = list[0].q;
            list[0].layout = kNN;
            s.after_own = true;
            s.a = d2;
            s.b = wp;
            s.M = T;
            s.N = a.dim;
            s.K = n;
            s.p.alpha = g.by_rows ? row_unscale : unscale;
            s.p.alpha_rows = g.by_rows;
            s.out[0] = last ? dh : sum;
            if (!first) {
                s.in[0] = sum;
                s.ins = 1;
                s.p.addend = last ? 2 : 1;
            }
            if (first && last)
                count = 1;
            else if ((rc = last ? run_product<kNN, kEpiStore>(s, dtype, c) : run_product<kNN, kEpiStoreF32>(s, dtype, c)) !=
                     GEMM_OK)
                return rc;
        }
        if (a.dw) {
            Product& s = list[count].q;
            s = Product();
            list[count++].layout = kTN;
            s.a = d;
            s.b = h;
            s.M = n;
            s.N = a.dim;
            s.K = T;
            s.p.alpha = unscale;
            s.out[0] = mat16(static_cast<char*>(a.dw) + (size_t)v0 * a.lddw * 2, n, a.dim, a.lddw);
        }
        if ((rc = run_grads(list, count, dtype, c)) != GEMM_OK) return rc;
    }
    return GEMM_OK;
}

int grad_clip_workspace(long long tensors, size_t* bytes) {
    if (!bytes) return GEMM_ERR_NULL;
    if (tensors < 0 || tensors > (1ll << 40)) return GEMM_ERR_DIM;
    const size_t launches = tensors <= kClipSmall ? 1 : (size_t)((tensors + kClipBig - 1) / kClipBig);
    *bytes = launches * kClipMaxBlocks * sizeof(float);
    return GEMM_OK;
}

int grad_clip(const grad_clip_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const grad_clip_args& a = *args;
    size_t need = 0;
    int rc = grad_clip_workspace(a.tensors, &need);
    if (rc != GEMM_OK) return rc;
    if (!(a.max_norm >= 0) || !(a.eps >= 0)) return GEMM_ERR_CONFIG;
    if (a.tensors > 0 && (!a.src || !a.dst || !a.count || !a.dtype)) return GEMM_ERR_NULL;
    if ((uintptr_t)a.norm & 3) return GEMM_ERR_ALIGN;
    long long entries = 0;
    for (long long i = 0; i < a.tensors; ++i) {
        if (a.count[i] < 0 || a.count[i] > (1ll << 44)) return GEMM_ERR_DIM;
        if (a.dtype[i] < LAYER_F16 || a.dtype[i] > LAYER_F32) return GEMM_ERR_DTYPE;
        if (a.count[i] == 0) continue;
        if (!a.src[i] || !a.dst[i]) return GEMM_ERR_NULL;
        const int b = a.dtype[i] == LAYER_F32 ? 4 : 2;
        if (((uintptr_t)a.src[i] | (uintptr_t)a.dst[i]) & (b - 1)) return GEMM_ERR_ALIGN;
        if (a.src[i] != a.dst[i]) {
            const Span s[] = {span_of(a.src[i], (uint64_t)a.count[i] * b)}, d[] = {span_of(a.dst[i], (uint64_t)a.count[i] * b)};
            if (overlaps(d, 1, s, 1)) return GEMM_ERR_ALIAS;
        }
        entries += a.count[i];
        if (entries > (1ll << 44)) return GEMM_ERR_DIM;
    }
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, need)) != GEMM_OK) return rc;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    return a.tensors <= kClipSmall ? run_clip<kClipSmall>(a, entries, c) : run_clip<kClipBig>(a, entries, c);
}

}  // extern "C"
