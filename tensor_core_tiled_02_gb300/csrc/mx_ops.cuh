// Host side of the norm and of the microscaled operands (include/mx_ops.h): argument
// checks, tensor maps, workspaces and launches.  Part of the library's one translation
// unit (tcgemm.cu), behind layer_ops.cuh, whose checks and launches it shares.
#pragma once

#include "mx_ops.h"

#include "mx_linear_kernel.cuh"
#include "mx_quant_kernel.cuh"
#include "norm_kernel.cuh"

namespace {

// A microscaled matrix as the caller describes it.
struct Mx {
    const void *data, *scale;
    long long rows, cols, ld;
    int fmt;
};

long long mx_blocks(const Mx& m) { return ceil_div(m.cols, kMxBlock); }
long long mx_width(const Mx& m) { return mx_blocks(m) * mx_block_bytes(m.fmt); }
Mat mx_data(const Mx& m) { return Mat{m.data, m.rows, mx_width(m), m.ld, 1}; }
uint64_t mx_scale_bytes(const Mx& m) { return (uint64_t)ceil_div(m.rows, 128) * ceil_div(m.cols, 128) * 512; }
Span mx_scale_span(const Mx& m) { return span_of(m.scale, mx_scale_bytes(m)); }

int check_mx(const Mx& m) {
    if (m.rows == 0 || m.cols == 0) return GEMM_OK;
    if (!m.data || !m.scale) return GEMM_ERR_NULL;
    if ((uintptr_t)m.scale & 15) return GEMM_ERR_ALIGN;
    return check_mat(mx_data(m));
}

int check_format(long long format) { return format == MX_E4M3 || format == MX_E2M1 ? GEMM_OK : GEMM_ERR_CONFIG; }

// dtype and format as compile-time tags.
template <typename F>
int with_types(long long dtype, long long format, F&& f) {
    using std::integral_constant;
    if (dtype == LAYER_BF16)
        return format == MX_E2M1 ? f(integral_constant<int, kBF16>{}, integral_constant<int, kE2M1>{})
                                 : f(integral_constant<int, kBF16>{}, integral_constant<int, kE4M3>{});
    return format == MX_E2M1 ? f(integral_constant<int, kF16>{}, integral_constant<int, kE2M1>{})
                             : f(integral_constant<int, kF16>{}, integral_constant<int, kE4M3>{});
}

// Shared memory that small blocks ask for without need: a kernel on CTA pairs leaves under 2 KB of
// an SM, so no norm or quantisation lies beside it (MxPairLayout).  Times are the same with and
// without.
constexpr int kNotBesidePairs = 2048;

// ---- norm ---------------------------------------------------------------------------------

template <int DT, int V, int OUT>
int run_norm_rows(const NormParams& p, int threads, const Ctx& c) {
    const int rows = p.group == 32 ? threads / 32 : 1;
    return launch_pdl(rms_norm_kernel<DT, V, OUT>, dim3(ceil_div(p.tokens, rows)), threads, kNotBesidePairs, 1, c.stream, p);
}

// Threads that share a row, and vectors of eight columns each has.
template <int DT, int OUT>
int run_norm(NormParams p, const Ctx& c) {
    const int vectors = ceil_div(p.dim, 8);
    if (vectors > 4 * 1024)
        return launch_pdl(rms_norm_long_kernel<DT, OUT>, dim3(p.tokens), 1024, kNotBesidePairs, 1, c.stream, p);
    // One vector a thread while all rows' threads are resident at once, else two, as a block
    // takes at most 1024 threads (with residual, one, two and four: 304 x 4096 2.7, 2.9 and 3.6
    // us; 512 x 8192 7.6, 6.7 and 6.9; 2048 x 4096 12.3, 10.8 and 12.3; 8192 x 4096 45.0, 42.0
    // and 42.8; into 8 bits 2000 x 4096 13.8, 12.3 and 12.8, 8192 x 4096 49.2, 42.0 and 40.1).
    int v = (long long)p.tokens * vectors <= 2048ll * c.dev->sms ? 1 : 2;
    while (vectors > 1024 * v) v *= 2;
    p.group = ceil_div(ceil_div(vectors, v), 32) * 32;
    const int threads = p.group == 32 ? 128 : p.group;
    switch (v) {
        case 1: return run_norm_rows<DT, 1, OUT>(p, threads, c);
        case 2: return run_norm_rows<DT, 2, OUT>(p, threads, c);
        default: return run_norm_rows<DT, 4, OUT>(p, threads, c);
    }
}

struct NormGradPlan {
    int threads, per_sm, blocks;
    size_t bytes;
};

// Two vectors of eight columns a thread, and as many blocks on an SM as make 512 threads.
NormGradPlan norm_grad_plan(const rms_norm_grad_args& a) {
    NormGradPlan g{};
    const int vectors = ceil_div(a.dim, 8);
    int threads = 64;
    while (threads < 2048 && 2 * threads < vectors) threads *= 2;
    g.threads = threads > 1024 ? 0 : threads;  // 0: long rows
    g.per_sm = threads >= 512 ? 1 : 512 / threads;
    // long rows: four blocks an SM over the columns and shares of the rows
    const int most = threads > 1024 ? std::max(8, 4 * kNormSms / ceil_div(a.dim, 2048)) : g.per_sm * kNormSms;
    g.blocks = a.tokens < most ? (int)a.tokens : most;
    g.bytes = a.dweight ? align256((size_t)g.blocks * pad8(a.dim) * 4) : 0;
    return g;
}

template <int DT, int DEPTH, int THREADS, int BLOCKS>
int run_norm_grad_rows(const NormGradParams& p, const NormGradPlan& g, const Ctx& c) {
    auto kern = rms_norm_grad_kernel<DT, DEPTH, THREADS, BLOCKS>;
    constexpr int kSmem = DEPTH * 3 * 2 * 16 * THREADS;
    static std::atomic<bool> ready[kMaxDevices];
    const int rc = ensure_smem_limit(kern, kSmem, ready[c.ordinal]);
    return rc != GEMM_OK ? rc : launch_pdl(kern, dim3(g.blocks), THREADS, kSmem, 1, c.stream, p);
}

template <int DT>
int run_norm_grad(const NormGradParams& p, const NormGradPlan& g, void* dweight, const Ctx& c) {
    int rc = GEMM_OK;
    switch (g.threads) {
        case 64: rc = run_norm_grad_rows<DT, 4, 64, 8>(p, g, c); break;
        case 128: rc = run_norm_grad_rows<DT, 4, 128, 4>(p, g, c); break;
        case 256: rc = run_norm_grad_rows<DT, 4, 256, 2>(p, g, c); break;
        case 512: rc = run_norm_grad_rows<DT, 4, 512, 1>(p, g, c); break;
        case 1024: rc = run_norm_grad_rows<DT, 2, 1024, 1>(p, g, c); break;
        default:
            // the column sums first: dx may be written over dy
            if (dweight)
                rc = launch_pdl(rms_norm_grad_columns_kernel<DT>, dim3(ceil_div(p.dim, 2048), g.blocks), 256, kNotBesidePairs, 1, c.stream, p);
            if (rc == GEMM_OK && p.dx) rc = launch_pdl(rms_norm_grad_long_kernel<DT>, dim3(p.tokens), 1024, kNotBesidePairs, 1, c.stream, p);
    }
    if (rc == GEMM_OK && dweight)
        rc = launch_pdl(rms_norm_weight_sum_kernel<DT>, dim3(ceil_div(p.dim, 32)), 1024, 0, 1, c.stream, p, dweight, g.blocks);
    return rc;
}

// ---- linear layer -------------------------------------------------------------------------

// `rows` rows of one K step of a microscaled matrix, 128-byte swizzled.
int encode_mx_data(CUtensorMap* out, const Mx& m, uint32_t rows) {
    cuuint64_t dims[2] = {(cuuint64_t)mx_width(m), (cuuint64_t)m.rows};
    cuuint64_t strides[1] = {(cuuint64_t)m.ld};
    cuuint32_t box[2] = {kMxStepBytes, rows}, estr[2] = {1, 1};
    return g_encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(m.data), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? GEMM_OK
               : GEMM_ERR_TMAP;
}

// Its scales: a row of tiles a row, in words; a K step is one tile or two.
int encode_mx_scale(CUtensorMap* out, const Mx& m) {
    const long long k_tiles = ceil_div(m.cols, 128);
    cuuint64_t dims[2] = {(cuuint64_t)k_tiles * 128, (cuuint64_t)ceil_div(m.rows, 128)};
    cuuint64_t strides[1] = {(cuuint64_t)k_tiles * 512};
    cuuint32_t box[2] = {(cuuint32_t)mx_step_tiles(m.fmt) * 128, 1}, estr[2] = {1, 1};
    return g_encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(m.scale), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? GEMM_OK
               : GEMM_ERR_TMAP;
}

struct MxProduct {
    Mx x, w;
    MxEpilogue e;
};

struct MxSkinnyPlan {
    int nt, t_tiles, tiles, split, slots, stage_bytes, smem, scale_col, tmem_cols, k_steps;
};

MxSkinnyPlan mx_skinny_plan(const MxProduct& q, DeviceInfo& dev) {
    const int sms = dev.sms;
    MxSkinnyPlan g{};
    const int fmt = q.x.fmt;
    // tokens from multiples of 128 on: there the tiles of their scales begin
    g.t_tiles = ceil_div(q.x.rows, 128);
    g.nt = g.t_tiles > 1 ? 128 : ceil_div(q.x.rows, 16) * 16;
    g.tiles = ceil_div(q.w.rows, 128) * g.t_tiles;
    g.k_steps = ceil_div(mx_width(q.x), kMxStepBytes);
    g.stage_bytes = (128 + g.nt) * kMxStepBytes + 1024 * mx_step_tiles(fmt);
    g.scale_col = (g.nt + 31) / 32 * 32;
    const int cols = g.scale_col + 16 * mx_step_tiles(fmt);
    g.tmem_cols = cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
    // Split along K until two SMs in three are busy, or four in five while a CTA still has
    // more than 24 steps (one token, K = 4096, N = 14336: 112 and 224 CTAs 7.9 and 8.5 us in
    // 4 bits, 16 steps; 13.2 and 12.9 in 8 bits, 32).
    g.split = 1;
    for (int s = 2; s <= kMaxSplit && 2 * s <= g.k_steps; ++s) {
        if (g.tiles * g.split >= (ceil_div(g.k_steps, g.split) > 24 ? sms * 4 / 5 : sms * 2 / 3)) break;
        g.split = s;
    }
    // Two CTAs fill an SM, so that the next launch's find room beside this one's (one token,
    // K = N = 4096, 8 bits: 6.5 us, 7.2 with the whole SM).  Larger tiles take all of it where
    // each has an SM to itself, for a ring of more than three steps (128 tokens, the same: 11.7
    // and 10.8), and all clusters fit at once (a cluster's CTAs share a GPC: of 48 clusters of
    // three some wait for others, 300 tokens, 4096 x 2048, 4 bits 14.7 us).
    const int fixed = 1024 + 8 * (2 * kMxSkinnySlots + 1) + 16;
    const bool alone = g.nt > 48 && g.tiles * g.split <= sms &&
                       (g.split == 1 || g.tiles <= (g.split == 2 ? max_pairs_of(dev) : max_clusters_of(dev, g.split)));
    g.smem = alone ? kSmemLimit : kSkinnyTwoSmem;
    g.slots = (g.smem - fixed) / g.stage_bytes;
    if (g.slots > kMxSkinnySlots) g.slots = kMxSkinnySlots;
    return g;
}

// Nanoseconds a product is expected to take, to choose between the kernels; memory at 6.5 bytes a
// picosecond.  The kernel for few tokens is not persistent: each generation of its CTAs pays all
// of a CTA's time again, which is a fixed part, the tokens' way through shared memory (their own
// share of them twice over with a residual) and 115 bytes a nanosecond of operands; two CTAs on
// an SM take 1.5 times as long as one.  Splits meet once.  A pair takes 334 a step; between two
// tiles it waits some 1540 for the columns its accumulators share, and a residual takes 5700 a
// tile that shorter products do not hide.
// (Against the better of the two kernels on 1940 products, 1 to 8192 tokens, K from 64 to 14336
// and N to 16384, either format, with a residual and without: 0.04 % lost on average, 10 % at
// worst; 8192 tokens, K = 64, N = 9216 33 us on pairs, 104 on the other, 81 and 276 with a
// residual.  499 others, K from 32 and N to 60000: 0.2 % and 13 %.  With a CTA's time charged
// once whatever their number the 1940 lost 21 % and 281 %.)
long long mx_product_bytes(const MxProduct& q) {
    const long long outputs = q.e.residual ? 2 : 1;
    return q.w.rows * mx_width(q.w) + q.x.rows * (mx_width(q.x) + 2 * outputs * q.w.rows);
}

long long mx_skinny_ns(const MxProduct& q, const MxSkinnyPlan& g, int sms) {
    const long long ctas = (long long)g.tiles * g.split, full = ctas / (2 * sms), rest = ctas % (2 * sms);
    const long long halves = 3 * full + (rest > sms ? 3 : rest > 0 ? 2 : 0);  // in units of half a lone CTA's time
    const long long cta = 320 + 25 * g.nt + (q.e.residual ? 53 * g.nt / g.split : 0) + (long long)ceil_div(g.k_steps, g.split) * g.stage_bytes / 115;
    const long long steps = 2400 + (g.split > 1 ? 1050 : 0) + halves * cta / 2;
    const long long memory = 3500 + mx_product_bytes(q) * 10 / 65000;
    return steps > memory ? steps : memory;
}

long long mx_pair_ns(const MxProduct& q, int pairs, int k_steps) {
    const long long tiles = (long long)ceil_div(q.x.rows, 256) * ceil_div(q.w.rows, 256);
    const long long waves = (tiles + pairs - 1) / pairs, tile = k_steps * 334ll;
    const long long steps = 4200 + (q.e.residual ? 2000 : 0) + tile + (waves - 1) * std::max(tile + 1540, q.e.residual ? 5700ll : 0ll);
    const long long memory = 4500 + mx_product_bytes(q) * 10 / 65000;
    return steps > memory ? steps : memory;
}

template <int FMT, int DT>
int run_mx_skinny(const MxProduct& q, const MxSkinnyPlan& g, const Ctx& c) {
    MxSkinnyMaps tm;
    std::memset(&tm, 0, sizeof(tm));
    int rc = encode_mx_data(&tm.x, q.x, g.nt);
    if (rc == GEMM_OK) rc = encode_mx_data(&tm.w, q.w, 128);
    if (rc != GEMM_OK) return rc;
    MxSkinnyParams p;
    std::memset(&p, 0, sizeof(p));
    p.T = (int)q.x.rows;
    p.N = (int)q.w.rows;
    p.nt = g.nt;
    p.t_tiles = g.t_tiles;
    p.blocks = (int)mx_blocks(q.x);
    p.k_steps = g.k_steps;
    p.split = g.split;
    p.slots = g.slots;
    p.stage_bytes = g.stage_bytes;
    p.tmem_cols = g.tmem_cols;
    p.scale_col = g.scale_col;
    p.xs = static_cast<const uint8_t*>(q.x.scale);
    p.ws = static_cast<const uint8_t*>(q.w.scale);
    p.k_tiles = ceil_div(q.x.cols, 128);
    p.e = q.e;
    p.wait_limit = c.wait_limit;
    p.inject = c.inject;
    auto kern = mx_skinny_kernel<FMT, DT>;
    static std::atomic<bool> ready[kMaxDevices];
    rc = ensure_smem_limit(kern, kSmemLimit, ready[c.ordinal]);
    if (rc != GEMM_OK) return rc;
    return launch_pdl(kern, dim3(g.tiles * g.split), kThreads, g.smem, g.split, c.stream, tm, p);
}

template <int FMT, int DT>
int run_mx_pair(const MxProduct& q, const Ctx& c) {
    using L = MxPairLayout<FMT>;
    MxMaps tm;
    std::memset(&tm, 0, sizeof(tm));
    int rc = encode_mx_data(&tm.x, q.x, 128);
    if (rc == GEMM_OK) rc = encode_mx_data(&tm.w, q.w, 128);
    if (rc == GEMM_OK) rc = encode_mx_scale(&tm.xs, q.x);
    if (rc == GEMM_OK) rc = encode_mx_scale(&tm.ws, q.w);
    constexpr int dtype = DT == kBF16 ? LAYER_BF16 : LAYER_F16;
    if (rc == GEMM_OK) rc = encode_out(&tm.y, mat16(q.e.y, q.x.rows, q.w.rows, q.e.ldy), dtype, 32);
    if (rc == GEMM_OK && q.e.residual) rc = encode_mat(&tm.residual, mat16(q.e.residual, q.x.rows, q.w.rows, q.e.ldr), dtype, 64, 32);
    if (rc != GEMM_OK) return rc;
    MxPairParams p;
    std::memset(&p, 0, sizeof(p));
    p.M = (int)q.x.rows;
    p.N = (int)q.w.rows;
    p.tiles_m = ceil_div(q.x.rows, 256);
    p.tiles_n = ceil_div(q.w.rows, 256);
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    p.blocks = (int)mx_blocks(q.x);
    p.k_steps = ceil_div(mx_width(q.x), kMxStepBytes);
    p.raster_group = 8;
    p.e = q.e;
    p.wait_limit = c.wait_limit;
    p.inject = c.inject;
    auto kern = mx_pair_kernel<FMT, DT>;
    static std::atomic<bool> ready[kMaxDevices];
    rc = ensure_smem_limit(kern, L::kSmem, ready[c.ordinal]);
    if (rc != GEMM_OK) return rc;
    const int pairs = max_pairs_of(*c.dev);
    return launch_pdl(kern, dim3(2 * (int)(tiles < pairs ? tiles : pairs)), L::kThreads, L::kSmem, 2, c.stream, tm, p);
}

template <int FMT, int DT>
int run_mx_product(const MxProduct& q, const Ctx& c) {
    // (more tiles than a grid counts: no matrix that fits this GPU has them)
    if ((long long)ceil_div(q.x.rows, 128) * ceil_div(q.w.rows, 128) > INT_MAX / kMaxSplit) return GEMM_ERR_DIM;
    const MxSkinnyPlan g = mx_skinny_plan(q, *c.dev);
    if (mx_skinny_ns(q, g, c.dev->sms) <= mx_pair_ns(q, max_pairs_of(*c.dev), g.k_steps)) return run_mx_skinny<FMT, DT>(q, g, c);
    return run_mx_pair<FMT, DT>(q, c);
}

int check_dtype16(long long dtype) { return check_dtype_act(dtype, LAYER_ACT_NONE); }

}  // namespace

extern "C" {

int rms_norm_forward(const rms_norm_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const rms_norm_args& a = *args;
    int rc = check_dtype16(a.dtype);
    if (rc != GEMM_OK) return rc;
    if ((a.data || a.scale) && (rc = check_format(a.format)) != GEMM_OK) return rc;
    if (!(a.eps >= 0.0)) return GEMM_ERR_CONFIG;
    if (!dims_ok({a.dim}, a.tokens)) return GEMM_ERR_DIM;
    if (a.tokens == 0) return GEMM_OK;
    const Mat x = mat16(a.x, a.tokens, a.dim, a.ldx), r = mat16(a.residual, a.tokens, a.dim, a.ldr);
    const Mat h = mat16(a.h, a.tokens, a.dim, a.ldh), y = mat16(a.y, a.tokens, a.dim, a.ldy);
    const Mx m{a.data, a.scale, a.tokens, a.dim, a.ldd, (int)a.format};
    if (!a.residual != !a.h || (!a.y && !a.data) || !a.data != !a.scale || !a.weight) return GEMM_ERR_NULL;
    if ((rc = check_mat(x)) != GEMM_OK) return rc;
    if (a.residual && (rc = check_all({r, h})) != GEMM_OK) return rc;
    if (a.y && (rc = check_mat(y)) != GEMM_OK) return rc;
    if (a.data && (rc = check_mx(m)) != GEMM_OK) return rc;
    if ((uintptr_t)a.weight & 15 || (uintptr_t)a.rstd & 3) return GEMM_ERR_ALIGN;
    const bool over_x = a.h == a.x && a.ldh == a.ldx, over_r = a.h == a.residual && a.ldh == a.ldr;
    const Span none{0, 0};
    const Span xs = span_of(x), rs = span_of(r), hs = span_of(h), ws = span_of(a.weight, (uint64_t)a.dim * 2);
    const Span others[] = {span_of(y), a.data ? span_of(mx_data(m)) : none, a.data ? mx_scale_span(m) : none,
                           span_of(a.rstd, (uint64_t)a.tokens * 4)};
    const Span all_read[] = {xs, rs, hs, ws};
    if (overlaps(others, 4, all_read, 4)) return GEMM_ERR_ALIAS;
    const Span h_read[] = {over_x ? none : xs, over_r ? none : rs, ws};
    if (overlaps(&hs, 1, h_read, 3)) return GEMM_ERR_ALIAS;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    NormParams p{};
    p.x = a.x;
    p.residual = a.residual;
    p.weight = a.weight;
    p.h = a.h;
    p.y = a.y;
    p.data = static_cast<uint8_t*>(a.data);
    p.scale = static_cast<uint32_t*>(a.scale);
    p.rstd = a.rstd;
    p.ldx = a.ldx;
    p.ldr = a.ldr;
    p.ldh = a.ldh;
    p.ldy = a.ldy;
    p.ldd = a.ldd;
    p.tokens = (int)a.tokens;
    p.dim = (int)a.dim;
    p.eps = (float)a.eps;
    if (!a.data) return a.dtype == LAYER_BF16 ? run_norm<kBF16, kNormRow>(p, c) : run_norm<kF16, kNormRow>(p, c);
    return with_types(a.dtype, a.format, [&](auto dt, auto fmt) {
        return run_norm<decltype(dt)::value, decltype(fmt)::value == kE4M3 ? kNormE4M3 : kNormE2M1>(p, c);
    });
}

int rms_norm_backward_workspace(const rms_norm_grad_args* args, size_t* bytes) {
    if (!args || !bytes) return GEMM_ERR_NULL;
    const int rc = check_dtype16(args->dtype);
    if (rc != GEMM_OK) return rc;
    if (!dims_ok({args->dim}, args->tokens)) return GEMM_ERR_DIM;
    *bytes = norm_grad_plan(*args).bytes;
    return GEMM_OK;
}

int rms_norm_backward(const rms_norm_grad_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const rms_norm_grad_args& a = *args;
    int rc = check_dtype16(a.dtype);
    if (rc != GEMM_OK) return rc;
    if (!dims_ok({a.dim}, a.tokens)) return GEMM_ERR_DIM;
    const Mat dy = mat16(a.dy, a.tokens, a.dim, a.lddy), h = mat16(a.h, a.tokens, a.dim, a.ldh);
    const Mat dh = mat16(a.dh, a.tokens, a.dim, a.lddh), dx = mat16(a.dx, a.tokens, a.dim, a.lddx);
    if (!a.weight || (a.tokens > 0 && !a.rstd)) return GEMM_ERR_NULL;
    if ((rc = check_all({dy, h})) != GEMM_OK) return rc;
    if (a.dh && (rc = check_mat(dh)) != GEMM_OK) return rc;
    if (a.dx && (rc = check_mat(dx)) != GEMM_OK) return rc;
    if (((uintptr_t)a.weight & 15) || ((uintptr_t)a.rstd & 3) || ((uintptr_t)a.dweight & 1)) return GEMM_ERR_ALIGN;
    const NormGradPlan g = norm_grad_plan(a);
    if (a.tokens > 0 && (rc = check_workspace(a.workspace, a.workspace_bytes, g.bytes)) != GEMM_OK) return rc;
    const bool over_dy = a.dx == a.dy && a.lddx == a.lddy, over_dh = a.dx == a.dh && a.lddx == a.lddh;
    const Span none{0, 0};
    const Span dys = span_of(dy), hs = span_of(h), dhs = span_of(dh), dxs = span_of(dx);
    const Span ws = span_of(a.weight, (uint64_t)a.dim * 2), ss = span_of(a.rstd, (uint64_t)a.tokens * 4);
    const Span others[] = {span_of(a.dweight, (uint64_t)a.dim * 2), span_of(g.bytes ? a.workspace : nullptr, g.bytes)};
    const Span all_read[] = {dys, hs, dhs, dxs, ws, ss};
    if (overlaps(others, 2, all_read, 6)) return GEMM_ERR_ALIAS;
    const Span dx_read[] = {over_dy ? none : dys, hs, over_dh ? none : dhs, ws, ss};
    if (overlaps(&dxs, 1, dx_read, 5)) return GEMM_ERR_ALIAS;
    if (!a.dx && !a.dweight) return GEMM_OK;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    if (a.tokens == 0) return a.dweight ? zero_mat(Mat{a.dweight, 1, a.dim, a.dim, 2}, c) : GEMM_OK;
    NormGradParams p{};
    p.dy = a.dy;
    p.h = a.h;
    p.weight = a.weight;
    p.dh = a.dh;
    p.rstd = a.rstd;
    p.dx = a.dx;
    p.partial = a.dweight ? static_cast<float*>(a.workspace) : nullptr;
    p.lddy = a.lddy;
    p.ldh = a.ldh;
    p.lddh = a.lddh;
    p.lddx = a.lddx;
    p.tokens = (int)a.tokens;
    p.dim = (int)a.dim;
    return a.dtype == LAYER_BF16 ? run_norm_grad<kBF16>(p, g, a.dweight, c) : run_norm_grad<kF16>(p, g, a.dweight, c);
}

int mx_quantize(const mx_quantize_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const mx_quantize_args& a = *args;
    int rc = check_dtype16(a.dtype);
    if (rc != GEMM_OK || (rc = check_format(a.format)) != GEMM_OK) return rc;
    if (a.transpose != 0 && a.transpose != 1) return GEMM_ERR_CONFIG;
    // either of the two may be the number of tokens
    if (!dims_ok({}, a.rows) || !dims_ok({}, a.cols)) return GEMM_ERR_DIM;
    if (a.rows == 0 || a.cols == 0) return GEMM_OK;
    const Mat x = mat16(a.x, a.rows, a.cols, a.ldx);
    const Mx m{a.data, a.scale, a.transpose ? a.cols : a.rows, a.transpose ? a.rows : a.cols, a.ldd, (int)a.format};
    if ((rc = check_mat(x)) != GEMM_OK || (rc = check_mx(m)) != GEMM_OK) return rc;
    const Span wr[] = {span_of(mx_data(m)), mx_scale_span(m)}, rd[] = {span_of(x)};
    if (overlaps(wr, 2, rd, 1)) return GEMM_ERR_ALIAS;
    MxQuantParams p{};
    p.x = a.x;
    p.data = static_cast<uint8_t*>(a.data);
    p.scale = static_cast<uint32_t*>(a.scale);
    p.ldx = a.ldx;
    p.ldd = a.ldd;
    p.rows = (int)a.rows;
    p.cols = (int)a.cols;
    p.groups = ceil_div(a.cols, a.transpose ? 128 : 256);
    const long long blocks = (long long)p.groups * ceil_div(a.rows, a.transpose ? 128 : 8 * kMxQuantRows);
    if (blocks > INT_MAX) return GEMM_ERR_DIM;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    return with_types(a.dtype, a.format, [&](auto dt, auto fmt) {
        constexpr int DT = decltype(dt)::value, FMT = decltype(fmt)::value;
        return a.transpose ? launch_pdl(mx_quantize_columns_kernel<DT, FMT>, dim3((unsigned)blocks), 256, 0, 1, c.stream, p)
                           : launch_pdl(mx_quantize_kernel<DT, FMT>, dim3((unsigned)blocks), 256, kNotBesidePairs, 1, c.stream, p);
    });
}

int mx_dequantize(const mx_dequantize_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const mx_dequantize_args& a = *args;
    int rc = check_dtype16(a.dtype);
    if (rc != GEMM_OK || (rc = check_format(a.format)) != GEMM_OK) return rc;
    if (!dims_ok({}, a.rows) || !dims_ok({}, a.cols)) return GEMM_ERR_DIM;
    if (a.rows == 0 || a.cols == 0) return GEMM_OK;
    const Mat x = mat16(a.x, a.rows, a.cols, a.ldx);
    const Mx m{a.data, a.scale, a.rows, a.cols, a.ldd, (int)a.format};
    if ((rc = check_mx(m)) != GEMM_OK || (rc = check_mat(x)) != GEMM_OK) return rc;
    const Span wr[] = {span_of(x)}, rd[] = {span_of(mx_data(m)), mx_scale_span(m)};
    if (overlaps(wr, 1, rd, 2)) return GEMM_ERR_ALIAS;
    MxValuesParams p{};
    p.data = static_cast<const uint8_t*>(a.data);
    p.scale = static_cast<const uint8_t*>(a.scale);
    p.x = a.x;
    p.ldd = a.ldd;
    p.ldx = a.ldx;
    p.rows = (int)a.rows;
    p.cols = (int)a.cols;
    p.groups = ceil_div(a.cols, 256);
    const long long blocks = (long long)p.groups * ceil_div(a.rows, 8 * kMxQuantRows);
    if (blocks > INT_MAX) return GEMM_ERR_DIM;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    return with_types(a.dtype, a.format, [&](auto dt, auto fmt) {
        return launch_pdl(mx_dequantize_kernel<decltype(dt)::value, decltype(fmt)::value>, dim3((unsigned)blocks), 256, kNotBesidePairs, 1, c.stream,
                          p);
    });
}

int mx_linear(const mx_linear_args* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_NULL;
    const mx_linear_args& a = *args;
    int rc = check_dtype_act(a.dtype, a.act);
    if (rc != GEMM_OK || (rc = check_format(a.format)) != GEMM_OK) return rc;
    if (!dims_ok({a.k, a.n}, a.tokens)) return GEMM_ERR_DIM;
    if (a.tokens == 0) return GEMM_OK;
    const Mx x{a.x, a.x_scale, a.tokens, a.k, a.ldx, (int)a.format}, w{a.w, a.w_scale, a.n, a.k, a.ldw, (int)a.format};
    const Mat y = mat16(a.y, a.tokens, a.n, a.ldy), r = mat16(a.residual, a.tokens, a.n, a.ldr);
    if ((rc = check_mx(x)) != GEMM_OK || (rc = check_mx(w)) != GEMM_OK || (rc = check_mat(y)) != GEMM_OK) return rc;
    if (r.p && (rc = check_mat(r)) != GEMM_OK) return rc;
    if ((uintptr_t)a.bias & 1) return GEMM_ERR_ALIGN;
    const bool in_place = r.p == y.p && a.ldr == a.ldy;
    const Span wr[] = {span_of(y)};
    const Span rd[] = {span_of(mx_data(x)), mx_scale_span(x), span_of(mx_data(w)), mx_scale_span(w),
                       span_of(a.bias, (uint64_t)a.n * 2), in_place ? Span{0, 0} : span_of(r)};
    if (overlaps(wr, 1, rd, 6)) return GEMM_ERR_ALIAS;
    Ctx c;
    if ((rc = open_ctx(c, stream)) != GEMM_OK) return rc;
    MxProduct q{x, w, {}};
    q.e.act = (int)a.act;
    q.e.bias = a.bias;
    q.e.residual = a.residual;
    q.e.y = a.y;
    q.e.ldr = a.ldr;
    q.e.ldy = a.ldy;
    return with_types(a.dtype, a.format, [&](auto dt, auto fmt) { return run_mx_product<decltype(fmt)::value, decltype(dt)::value>(q, c); });
}

#ifdef TCGEMM_CHECK
int mx_linear_check_times(const mx_linear_args* args, int sms, long long* few, long long* pairs) {
    if (!args || !few || !pairs) return GEMM_ERR_NULL;
    const mx_linear_args& a = *args;
    if (check_format(a.format) != GEMM_OK) return GEMM_ERR_CONFIG;
    if (!dims_ok({a.k, a.n}, a.tokens) || a.tokens < 1 || sms < 2) return GEMM_ERR_DIM;
    DeviceInfo dev;
    dev.sms = sms;
    dev.max_pairs = sms / 2;
    for (int s = 2; s <= kMaxSplit; ++s) dev.max_clusters[s] = std::max(1, fit_estimate(sms).clusters[s]);
    MxProduct q{Mx{a.x, a.x_scale, a.tokens, a.k, a.ldx, (int)a.format}, Mx{a.w, a.w_scale, a.n, a.k, a.ldw, (int)a.format}, {}};
    q.e.residual = a.residual;
    const MxSkinnyPlan g = mx_skinny_plan(q, dev);
    *few = mx_skinny_ns(q, g, sms);
    *pairs = mx_pair_ns(q, sms / 2, g.k_steps);
    return GEMM_OK;
}
#endif

}  // extern "C"
