// The layer operators' matrix product on CTA pairs: D = A B on 256 x 256 tiles
// (tcgen05.mma.cta_group::2, M = 256), fp16 or bf16 operands, each in either
// major order, fp32 accumulation in Tensor Memory, and the operator's own
// elementwise work in the epilogue, on the fp32 accumulator.
//
//   layout  A              B               products
//   NN      [M, K]         [K, N]          x w
//   NT      [M, K]         [N, K]          dy w^T, h W^T (vocabulary rows)
//   TN      [K, M]         [K, N]          x^T dy
//
//   epilogue        what it computes of the tile's values v
//   kEpiStore       y = act(alpha v + bias) + addend; keeps alpha v + bias on request.
//                   The addend is the residual, or the fp32 sum so far
//   kEpiGate        the tile's first 128 columns come from w_gate, the others
//                   from w_up (each CTA of the pair loads one of them), so a
//                   thread holds both g and u of an element: h = act(g) u
//   kEpiGateGrad    v = dh: dg = dh u act'(g), du = dh act(g), with g and u loaded
//   kEpiLossStats   v = logits: per row and tile the maximum and the sum of
//                   exp(v - maximum), and the target's logit; no logit is stored
//   kEpiLossStatsLong  the same for more than kPromote K steps: the tensor core's sums are
//                   added up in fp32 every kPromote steps
//   kEpiLossGrad    v = logits again: (exp(v - lse) - [column = target]) times the row's
//                   weight, in 16 bits, operand of the two products that follow
//   kEpiLossGradLong   the same with the logits summed as in kEpiLossStatsLong, so that
//                   they are those the lse was made of, to the bit: where a target's p is
//                   near 1, p - 1 is smaller than what the two ways of summing differ by
//
// Two operand pairs may follow one another along K (dx = dg Wg^T + du Wu^T is
// one product whose K is both halves): K steps from k_switch on read a[1], b[1].
//
// Bound by the tensor pipe at the sizes that matter: a 256 x 256 pair tile
// reads 32 KiB of operands per SM per 64 of K, 512 cycles of MMA.  Persistent
// pairs walk the tiles in the grouped raster of gemm_common.cuh; the TMEM
// accumulator is double-buffered, so a tile's epilogue (arithmetic of 15 to 40
// instructions an element on four warps) runs under the next tile's products.
// (Eight warps drain a tile sooner, but cost the products 2 %: 8192 tokens of the
// gated block at 4096 x 14336 1519 us on four, 1542 on eight.  Now 1510, 1911 TFLOP/s;
// 4096 tokens, 4096 x 14336 with bias and GELU 261.5 us, 1840 TFLOP/s.)  What an epilogue reads
// and writes moves by TMA through four 4 KiB buffers per warp (in place where it
// reads), leaving five 32 KiB stages.
//
// SPLIT (kEpiStore, few tiles): a cluster of 2 to 4 pairs shares a tile along K.
// Each CTA leaves its 128 rows of fp32 partials in its idle ring; then every
// pair drains a share of the tile's columns, summing the partials of its rows over
// distributed shared memory in rank order.  Nothing else hides that drain, so eight
// warps run it, two on each quarter of the rows.
//
// Roles as in gemm_pair_kernel.cuh: warp 0 loads, warp 1 issues MMAs (even CTA),
// the others drain; every wait is bounded and reports through the status word.
#pragma once

#include "layer_common.cuh"

namespace tcgemm {

enum LayerLayout { kNN = 0, kNT = 1, kTN = 2 };
enum LayerEpilogue {
    kEpiStore = 0,
    kEpiStoreF32 = 1,
    kEpiGate = 2,
    kEpiGateGrad = 3,
    kEpiLossStats = 4,
    kEpiLossGrad = 5,
    kEpiLossStatsLong = 6,
    kEpiLossGradLong = 7,
};

constexpr int kLayerMaxSplit = 4;
__host__ __device__ constexpr bool loss_long(int epi) { return epi == kEpiLossStatsLong || epi == kEpiLossGradLong; }
// loss_long: K steps (of 64) summed on the tensor core at a time.  It truncates as it adds: a
// logit whose terms all have one sign is low by 6e-9 of itself a unit of K in fp16 and by half
// that in bf16, up to 3.6e-6 and 3.4e-6 after these runs (1.2e-5 in fp16 after 2048; terms of
// random signs lose nothing on average).  Statistics in runs of 2048 took less: 1000 tokens,
// 2048 x 50021, fp16 133 us against 144; 4096 tokens, 4096 x 65536, bf16 1124 against 1140.
template <int DT>
constexpr int kPromote = DT == kF16 ? 8 : 16;

struct LayerMaps {
    CUtensorMap a[2], b[2];
    CUtensorMap out[3];
    CUtensorMap in[2];
};

struct LayerParams {
    int M, N;              // of the output (kEpiGate: N of h, half the product's)
    int tiles_m, tiles_n;
    int k_steps, k_switch; // 64-deep; steps >= k_switch read a[1], b[1] from their start
    int raster_group;
    int split;             // SPLIT: pairs sharing a tile along K
    int act;
    int addend;            // kEpiStore*: 0 none, 1 of the output's type, 2 fp32 under a 16-bit output
    int keep;              // kEpiStore: keep alpha v + bias in out[1]; kEpiGate: keep g and u in out[1], out[2];
                           // kEpiLossGrad*: the same with row_scale2 for row_scale in out[1]
    const void* bias;      // N values of the operands' type, or NULL
    const float* alpha;    // device scalar, or NULL for 1
    int alpha_rows;        // one alpha a row: [M]
    float2* stats;         // kEpiLossStats: [ceil(N / 128)][M] (maximum, sum of exponentials)
    float* target_logit;   // kEpiLossStats: [M], written where the target's column is met
    const long long* target;  // kEpiLoss*: [M]
    int col0;              // kEpiLossGrad: vocabulary index of the tile grid's first column
    const float* lse;      // kEpiLossGrad: [M]
    const float* row_scale;// kEpiLossGrad: [M], 0 for a row that takes no part
    const float* row_scale2;
    void* tail_out[3];     // kEpiStore, kEpiGate: the outputs again, for columns from N & ~7 on (store_tail)
    long long tail_ld[3];
    long long wait_limit;
    int inject;
};

constexpr int kTileN = 256;  // a pair tile's columns

template <int EPI, bool SPLIT>
struct LayerPairLayout {
    static constexpr int kABytes = 128 * 64 * 2;         // this CTA's 128 rows of one K step
    static constexpr int kBBytes = (kTileN / 2) * 64 * 2;    // this CTA's half of the columns
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kWarps = SPLIT || loss_long(EPI) ? 8 : 4;  // epilogue warps
    static constexpr int kThreads = 64 + 32 * kWarps;
    static constexpr int kWarpStaging = EPI == kEpiLossStats || EPI == kEpiLossStatsLong ? 0 : 65536 / kWarps;  // staging per epilogue warp
    // full[8], empty[8], tmem_full[2], tmem_empty[2], drain, aux[warps][2]
    static constexpr int kNumBars = 2 * kMaxStages + 5 + 2 * kWarps;
    static constexpr int kBiasBytes = kWarps * 64 * 2;   // 64 values per epilogue warp
    static constexpr int kFixedBytes = kWarps * kWarpStaging + kBiasBytes + ((kNumBars * 8 + 15) & ~15) + 16;
    static constexpr int kLimit = 232448;
    static constexpr int kFit = (kLimit - 1024 - kFixedBytes) / kStageBytes;
    static constexpr int kSlots = kFit < kMaxStages ? kFit : kMaxStages;
    static_assert(kSlots >= 5, "ring depth");
    static constexpr int kSmem = 1024 + kSlots * kStageBytes + kFixedBytes;
    static constexpr int kTmemCols = 2 * kTileN;             // two accumulators
    static constexpr int kOutN = EPI == kEpiGate ? kTileN / 2 : kTileN;      // output columns of a tile
    static constexpr int kChunk = EPI == kEpiStoreF32 || EPI == kEpiLossStats ? 32 : 64;  // columns drained at a time
};

__device__ __forceinline__ void layer_tile_coords(int t, const LayerParams& p, int& mb, int& nb) {
    const int g = p.raster_group;
    const int per_group = g * p.tiles_n;
    const int grp = t / per_group;
    const int first_m = grp * g;
    const int gm = min(p.tiles_m - first_m, g);
    const int r = t - grp * per_group;
    mb = first_m + r % gm;
    nb = r / gm;
    if (grp & 1) nb = p.tiles_n - 1 - nb;
}

// 16 bytes of this lane's row `lane` of a 32-row, 128-byte-swizzled buffer.
__device__ __forceinline__ uint32_t swz(uint32_t buf, int lane, int piece) {
    return buf + (uint32_t)(lane * 128) + ((uint32_t)(piece ^ (lane & 7)) << 4);
}

template <int LAY, int EPI, int DT, bool SPLIT>
__global__ void __launch_bounds__(LayerPairLayout<EPI, SPLIT>::kThreads, 1)
    layer_pair_kernel(const __grid_constant__ LayerMaps tm, const LayerParams p) {
    using L = LayerPairLayout<EPI, SPLIT>;
    constexpr bool kAMN = LAY == kTN, kBMN = LAY != kNT;
    constexpr int S = L::kSlots;
    constexpr int kHalf = kTileN / 2;
    static_assert(!SPLIT || (EPI == kEpiStore && S * L::kStageBytes >= 128 * kTileN * 4), "partials fit the ring");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    const uint32_t sA = base;
    const uint32_t sB = sA + S * L::kABytes;
    const uint32_t sC = sB + S * L::kBBytes;
    const uint32_t sBias = sC + L::kWarps * L::kWarpStaging;
    const uint32_t bar0 = sBias + L::kBiasBytes;
    const uint32_t misc = bar0 + ((L::kNumBars * 8 + 15) & ~15);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base_ptr + (misc - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + (misc - base) + 4);
#ifdef TCGEMM_CHECK
    if (misc + 16 > raw + ptx::dynamic_smem_size()) {
        if (threadIdx.x == 0) record_timeout(kSiteSmemBounds);
        return;
    }
#endif
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * kMaxStages + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 4);
    auto aux_bar = [&](int e, int set) { return bar0 + 8u * (2 * kMaxStages + 5 + 2 * e + set); };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t cta = ptx::cluster_ctarank();
    const uint32_t rank = cta & 1;         // in its pair: 0 issues the MMAs
    const uint32_t leader = cta & ~1u;
    const uint16_t both = (uint16_t)(3u << leader);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(tfull_bar(a), 1);
            ptx::mbar_init(tempty_bar(a), 2 * L::kWarps);  // every epilogue warp of both CTAs
        }
        ptx::mbar_init(drain_bar, 1);
        for (int i = 0; i < 2 * L::kWarps; ++i) ptx::mbar_init(aux_bar(i >> 1, i & 1), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tmap(&tm.a[0]);
        ptx::prefetch_tmap(&tm.b[0]);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr((const void*)tmem_slot), L::kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // the parts of the carve-up, for the bounds-check build's tests
    const uint32_t bars = (uint32_t)L::kNumBars * 8u, staging_all = (uint32_t)(L::kWarps * L::kWarpStaging);
    (void)bars, (void)staging_all;
    auto stage_ok = [&](int st) {
        return holds(bar0, bars, empty_bar(st), 8) && holds(bar0, bars, full_bar(st), 8) &&
               holds(sA, (uint32_t)(S * L::kABytes), sA + st * L::kABytes, L::kABytes) &&
               holds(sB, (uint32_t)(S * L::kBBytes), sB + st * L::kBBytes, L::kBBytes);
    };
    (void)stage_ok;

    // this cluster's tiles: cluster, cluster + clusters, ... (SPLIT: one), and its K steps [kb0, kb1)
    const int cluster = SPLIT ? (int)blockIdx.x / (2 * p.split) : (int)blockIdx.x >> 1;
    const int clusters = SPLIT ? (int)gridDim.x / (2 * p.split) : (int)gridDim.x >> 1;
    const int tiles = p.tiles_m * p.tiles_n;
    const int share = SPLIT ? (int)(cta >> 1) : 0;
    const int kb0 = SPLIT ? (int)((long long)p.k_steps * share / p.split) : 0;
    const int kb1 = SPLIT ? (int)((long long)p.k_steps * (share + 1) / p.split) : p.k_steps;

    bool split_met = false;
    (void)split_met;
    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        if (lane == 0 && p.inject == 0) {
            int stage = 0;
            uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
            bool ok = true;
            // the previous kernel's writes of the operands are done from here on
            ptx::grid_dependency_wait();
            ptx::grid_launch_dependents();
            for (int t = cluster; ok && t < tiles; t += clusters) {
                int mb, nb;
                layer_tile_coords(t, p, mb, nb);
                const int m0 = mb * 256 + (int)rank * 128;
                // kEpiGate: this CTA's columns are the tile's half of one weight
                const int n0 = EPI == kEpiGate ? nb * kHalf : nb * kTileN + (int)rank * kHalf;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!TC_CHECK(stage_ok(stage), kSiteSmemBounds)) {
                        ok = false;
                        break;
                    }
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.wait_limit, kSiteProducerEmpty)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb_local = full_bar(stage);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(fb_local, 2 * L::kStageBytes);
                    const uint32_t fb = ptx::mapa(fb_local, leader);
                    const int second = kb >= p.k_switch;
                    const int k0 = (second ? kb - p.k_switch : kb) * 64;
                    const CUtensorMap* ta = &tm.a[second];
                    const CUtensorMap* tb = &tm.b[EPI == kEpiGate ? (int)rank : second];
                    const uint32_t a = sA + stage * L::kABytes, b = sB + stage * L::kBBytes;
                    if constexpr (kAMN) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            ptx::tma_load_2d_pair(a + j * kBoxBytes, ta, fb, m0 + j * 64, k0);
                    } else {
                        ptx::tma_load_2d_pair(a, ta, fb, k0, m0);
                    }
                    if constexpr (kBMN) {
#pragma unroll
                        for (int j = 0; j < kHalf / 64; ++j)
                            ptx::tma_load_2d_pair(b + j * kBoxBytes, tb, fb, n0 + j * 64, k0);
                    } else {
                        ptx::tma_load_2d_pair(b, tb, fb, k0, n0);
                    }
                    issued_mask |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // both CTAs' bytes land before shared memory goes away
            if (rank == 0)
                for (int s = 0; s < S; ++s)
                    if (issued_mask & (1u << s)) wait_drain(full_bar(s), (issued_phase >> s) & 1u, p.wait_limit);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader only) ----------------
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = layer_idesc(DT, kAMN, kBMN, 256, kTileN);
            int stage = 0;
            uint32_t phase = 0;
            int tl = 0;
            bool ok = true;
            for (int t = cluster; ok && t < tiles; t += clusters) {
                // one accumulator a tile, or (loss_long) one every kPromote<DT> steps
                for (int ks = kb0, ke; ok && ks < kb1; ks = ke) {
                    ke = loss_long(EPI) ? min(kb1, ks + kPromote<DT>) : kb1;
                    const int acc = tl & 1;
                    const uint32_t aph = (tl >> 1) & 1;
                    ++tl;
                    if (!wait_bounded<true>(tempty_bar(acc), aph ^ 1u, abort_flag, p.wait_limit, kSiteMmaTmemEmpty)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kTileN);
                    if (!TC_CHECK(acc * kTileN + kTileN <= L::kTmemCols, kSiteTmemBounds)) {
                        ok = false;
                        break;
                    }
                    for (int kb = ks; kb < ke; ++kb) {
                        if (!TC_CHECK(stage_ok(stage), kSiteSmemBounds)) {
                            ok = false;
                            break;
                        }
                        if (!wait_bounded(full_bar(stage), phase, abort_flag, p.wait_limit, kSiteMmaFull)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        const uint64_t ad0 = operand_desc<kAMN>(sA + stage * L::kABytes);
                        const uint64_t bd0 = operand_desc<kBMN>(sB + stage * L::kBBytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_f16_ss_pair(d_tmem, ad0 + k * kSliceStep<kAMN>, bd0 + k * kSliceStep<kBMN>, idesc,
                                                 (kb - ks) | k);
                        ptx::mma_commit_pair_multicast(empty_bar(stage), both);
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    ptx::mma_commit_pair_multicast(tfull_bar(acc), both);
                }
            }
            ptx::mma_commit_pair(drain_bar);
            wait_drain(drain_bar, 0, p.wait_limit);
        }
    } else if constexpr (loss_long(EPI)) {
        // ---------------- loss, long K (both CTAs): 32 rows x 128 columns a warp ----------------
        // The sums of kPromote<DT> steps each are added up here in fp32, rounded to nearest, 128
        // columns a thread.
        const int ew = warp - 2, q = warp & 3, half = ew >> 2;
        const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 128);
        const uint32_t stg = sC + (uint32_t)(ew * L::kWarpStaging);
        (void)stg;
        ptx::grid_dependency_wait();
        ptx::grid_launch_dependents();
        int tl = 0;
        unsigned n_chunk = 0;  // kEpiLossGradLong: chunks of 64 columns stored; their two buffers alternate
        bool ok = true;
        for (int t = cluster; ok && t < tiles; t += clusters) {
            int mb, nb;
            layer_tile_coords(t, p, mb, nb);
            const int row0 = mb * 256 + (int)rank * 128 + q * 32, row = row0 + lane;
            const int x = nb * kTileN + half * 128;
            const bool mine = row0 < p.M && x < p.N;
            float lse = 0.0f, scale = 0.0f, scale2 = 0.0f;
            int tcol = -1;  // the target's column, relative to this warp's
            if (mine && row < p.M) {
                const long long tg = p.target[row] - p.col0 - x;
                if (tg >= 0 && tg < 128 && tg < p.N - x) tcol = (int)tg;
                if constexpr (EPI == kEpiLossGradLong) {
                    lse = p.lse[row];
                    scale = p.row_scale[row];
                    if (p.keep) scale2 = p.row_scale2[row];
                }
            }
            float v[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) v[i] = 0.0f;
            for (int ks = 0; ks < kb1; ks += kPromote<DT>, ++tl) {
                const int acc = tl & 1;
                ok = warp_wait(tfull_bar(acc), (tl >> 1) & 1, abort_flag, 4 * p.wait_limit, kSiteEpilogueTmemFull, lane);
                if (!ok) break;
                ptx::tc_fence_after();
                if (mine) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t w[32];
                        ptx::tmem_ld_32x32b_x32(lane_base + (uint32_t)(acc * kTileN + g * 32), w);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[g * 32 + i] += __uint_as_float(w[i]);
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0 && (t + clusters < tiles || ks + kPromote<DT> < kb1))
                    ptx::mbar_arrive_cluster(ptx::mapa(tempty_bar(acc), leader));
            }
            if (!ok || !mine) continue;
            if constexpr (EPI == kEpiLossStatsLong) {
                if (tcol >= 0) {
                    float picked = 0.0f;
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i == tcol) picked = v[i];
                    p.target_logit[row] = picked;
                }
                __syncwarp();
                if (p.N - x < 128) {  // columns from N on are no words
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i >= p.N - x) v[i] = -INFINITY;
                }
                float m0 = v[0], m1 = v[1];
#pragma unroll
                for (int i = 2; i < 128; i += 2) {
                    m0 = fmaxf(m0, v[i]);
                    m1 = fmaxf(m1, v[i + 1]);
                }
                const float m = fmaxf(m0, m1);
                // the difference before the factor: a maximum near the type's lowest times log2(e)
                // would overflow.  (While all is -inf the terms are exp(-inf - 0) = 0.)
                const float mf = m == -INFINITY ? 0.0f : m;
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 128; ++i) s[i & 3] += ex2_approx((v[i] - mf) * 1.4426950408889634f);
                if (row < p.M) p.stats[(size_t)(x >> 7) * p.M + row] = make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (x + c * 64 >= p.N) break;
                    // one of the two buffers in turn, or both
                    const uint32_t buf = p.keep ? stg : stg + (n_chunk & 1) * 4096u;
                    if (!TC_CHECK(holds(sC, staging_all, buf, p.keep ? 8192u : 4096u), kSiteSmemBounds)) break;
                    if (lane == 0) {
                        if (p.keep) ptx::bulk_wait_group_read<0>();
                        else ptx::bulk_wait_group_read<1>();  // the store two chunks ago has read its buffer
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float e[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int col = c * 64 + j * 8 + i;
                            e[i] = ex2_approx((v[col] - lse) * 1.4426950408889634f);
                            if (col == tcol) e[i] -= 1.0f;
                        }
                        // a row of weight 0 is 0 whatever its logits hold
                        auto put = [&](uint32_t to, float by) {
                            auto at = [&](int i) { return by == 0.0f ? 0.0f : e[i] * by; };
                            ptx::st_shared_v4(swz(to, lane, j), pack2<DT>(at(0), at(1)), pack2<DT>(at(2), at(3)),
                                              pack2<DT>(at(4), at(5)), pack2<DT>(at(6), at(7)));
                        };
                        put(buf, scale);
                        if (p.keep) put(buf + 4096, scale2);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_2d(&tm.out[0], buf, x + c * 64, row0);
                        if (p.keep) ptx::tma_store_2d(&tm.out[1], buf + 4096, x + c * 64, row0);
                        ptx::bulk_commit_group();
                    }
                    ++n_chunk;
                }
            }
        }
        if (EPI == kEpiLossGradLong && lane == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
    } else {
        // ---------------- epilogue (both CTAs): 32 rows a warp, all columns or (SPLIT) half ----------------
        const int ew = warp - 2;
        const int q = warp & 3;                  // TMEM lanes 32 q ..
        const int half = SPLIT ? ew >> 2 : 0;    // of the pair's share of columns
        const uint32_t stg = sC + (uint32_t)(ew * L::kWarpStaging);
        const uint32_t sbias = sBias + (uint32_t)(ew * 128);
        const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16);
        // the previous kernel's reads and writes of what this one touches are done from here on
        ptx::grid_dependency_wait();
        ptx::grid_launch_dependents();
        constexpr bool kLoads = EPI == kEpiStore || EPI == kEpiStoreF32 || EPI == kEpiGateGrad;
        const bool loads = kLoads && (EPI == kEpiGateGrad || p.addend != 0);
        float alpha = 1.0f;
        if constexpr (EPI == kEpiStore || EPI == kEpiStoreF32)
            if (p.alpha != nullptr && !p.alpha_rows) alpha = *p.alpha;

        // A chunk takes one buffer, or two where two matrices move (kEpiGate that keeps g and
        // u: three); while the staging holds two such sets they alternate, and the
        // next chunk's loads run under this one's work.
        constexpr bool kAlwaysTwo = EPI == kEpiGateGrad;
        const bool two_bufs = kAlwaysTwo || (EPI == kEpiStore && (p.keep || p.addend == 2)) || (EPI == kEpiLossGrad && p.keep);
        const bool one_set = (EPI == kEpiGate && p.keep) || (SPLIT && two_bufs);
        const bool four_sets = !SPLIT && !loads && !two_bufs && !one_set;  // nothing to load: all four in turn
        auto set_of = [&](unsigned n) {
            return one_set ? stg : four_sets ? stg + (n & 3) * 4096u : stg + (n & 1) * (two_bufs ? 8192u : 4096u);
        };
        auto wait_stores = [&]() {  // lane 0: the set about to be used is no longer read by a store
            if (one_set)
                ptx::bulk_wait_group_read<0>();
            else if (four_sets)
                ptx::bulk_wait_group_read<3>();
            else
                ptx::bulk_wait_group_read<1>();
        };
        // this warp's chunks of a tile, those with columns below N; rows from M on are no one's
        constexpr int kChunks = L::kOutN / L::kChunk;
        const int share0 = SPLIT ? kChunks * share / p.split : 0;
        const int share1 = SPLIT ? kChunks * (share + 1) / p.split : kChunks;
        const int mid = share0 + (share1 - share0 + 1) / 2;
        const int c0 = SPLIT && half ? mid : share0;
        auto chunk_end = [&](int nb) {
            return min(SPLIT && !half ? mid : share1, (p.N - nb * L::kOutN + L::kChunk - 1) / L::kChunk);
        };
        // the loads of one chunk (lane 0)
        auto issue_loads = [&](int row0, int x, unsigned n) {
            const uint32_t bar = aux_bar(ew, n & 1), buf = set_of(n);
            if constexpr (EPI == kEpiGateGrad) {
                ptx::mbar_arrive_expect_tx(bar, 8192);
                ptx::tma_load_2d(buf, &tm.in[0], bar, x, row0);
                ptx::tma_load_2d(buf + 4096, &tm.in[1], bar, x, row0);
            } else if (EPI == kEpiStore && p.addend == 2) {
                ptx::mbar_arrive_expect_tx(bar, 8192);
                ptx::tma_load_2d(buf, &tm.in[0], bar, x, row0);
                ptx::tma_load_2d(buf + 4096, &tm.in[0], bar, x + 32, row0);
            } else {
                ptx::mbar_arrive_expect_tx(bar, 4096);
                ptx::tma_load_2d(buf, &tm.in[0], bar, x, row0);
            }
        };
        unsigned n_chunk = 0;           // chunks this warp has drained: barrier n_chunk & 1, phase n_chunk >> 1
        bool pending = false;           // loads of chunk n_chunk are under way
        int tl = 0;
        for (int t = cluster; t < tiles; t += clusters) {
            int mb, nb;
            layer_tile_coords(t, p, mb, nb);
            const int acc = tl & 1;
            const uint32_t aph = (tl >> 1) & 1;
            ++tl;
            const int row0 = mb * 256 + (int)rank * 128 + q * 32;
            const int row = row0 + lane;
            const int n0 = nb * L::kOutN;
            const bool rows_here = row0 < p.M;
            const int c1 = rows_here ? chunk_end(nb) : 0;
            const bool last_tile = t + clusters >= tiles;
            if constexpr (kLoads) {
                if (loads && c0 < c1 && !pending) {
                    if (lane == 0) {
                        ptx::bulk_wait_group_read<0>();
                        issue_loads(row0, n0 + c0 * L::kChunk, n_chunk);
                    }
                    pending = true;
                }
            }
            // per-row values of the loss epilogues
            float lse = 0.0f, scale = 0.0f, scale2 = 0.0f, best = -INFINITY, sum = 0.0f;
            int tcol = -1;  // the target's column, relative to the tile grid
            if constexpr (EPI == kEpiLossStats || EPI == kEpiLossGrad) {
                if (row < p.M) {
                    const long long tg = p.target[row];
                    if (tg >= p.col0 && tg - p.col0 < p.N) tcol = (int)(tg - p.col0);
                    if constexpr (EPI == kEpiLossGrad) {
                        lse = p.lse[row];
                        scale = p.row_scale[row];
                        if (p.keep) scale2 = p.row_scale2[row];
                    }
                }
            }
            if constexpr (EPI == kEpiStore || EPI == kEpiStoreF32)
                if (p.alpha_rows) alpha = row < p.M ? p.alpha[row] : 0.0f;
            if (!warp_wait(tfull_bar(acc), aph, abort_flag, 4 * p.wait_limit, kSiteEpilogueTmemFull, lane)) break;
            ptx::tc_fence_after();
            const uint32_t trow = lane_base + (uint32_t)(acc * kTileN);
            auto hand_back = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0 && !last_tile) ptx::mbar_arrive_cluster(ptx::mapa(tempty_bar(acc), leader));
            };
            if constexpr (SPLIT) {
                // this CTA's partial into its ring (idle: every load was consumed by an MMA, every
                // MMA is complete): 16-byte groups of four columns, [group][row], read below
                for (int c = half * (kTileN / 64); c < (half + 1) * (kTileN / 64); ++c) {  // 32 columns
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(trow + c * 32, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        ptx::st_shared_v4(sA + (uint32_t)(((c * 8 + g) * 128 + q * 32 + lane) * 16), v[4 * g], v[4 * g + 1],
                                          v[4 * g + 2], v[4 * g + 3]);
                }
                // every epilogue thread of the cluster; the other warps arrived at once
                __syncwarp();
                ptx::cluster_arrive();
                ptx::cluster_wait();
                split_met = true;
            }
            if (!SPLIT && c0 >= c1) hand_back();
            bool failed = false;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                const int x = n0 + c * L::kChunk;
                const uint32_t buf0 = set_of(n_chunk), buf1 = buf0 + 4096;
                if constexpr (EPI == kEpiLossStats) {
                    __syncwarp();  // the lanes part where one of them meets its target
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(trow + c * 32, v);
                    ptx::tmem_ld_wait();
                    if (!SPLIT && c == c1 - 1) hand_back();
                    if (p.N - x < 32) {  // columns from N on are no words
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i >= p.N - x) v[i] = 0xFF800000u;  // -inf
                    }
                    float m = best;
#pragma unroll
                    for (int i = 0; i < 32; ++i) m = fmaxf(m, __uint_as_float(v[i]));
                    sum *= best == m ? 1.0f : ex2_approx((best - m) * 1.4426950408889634f);
                    // the difference before the factor: a maximum near the type's lowest times log2(e)
                    // would overflow.  (While all is -inf the terms are exp(-inf - 0) = 0.)
                    const float mf = m == -INFINITY ? 0.0f : m;
                    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        s0 += ex2_approx((__uint_as_float(v[i]) - mf) * 1.4426950408889634f);
                        s1 += ex2_approx((__uint_as_float(v[i + 1]) - mf) * 1.4426950408889634f);
                    }
                    sum += s0 + s1;
                    best = m;
                    if ((c & 3) == 3 || c == c1 - 1) {  // a part of 128 columns is whole
                        if (row < p.M) p.stats[(size_t)(x >> 7) * p.M + row] = make_float2(best, sum);
                        best = -INFINITY;
                        sum = 0.0f;
                    }
                    const int rel = tcol - x;
                    if (rel >= 0 && rel < 32) {
                        float tv = 0.0f;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i == rel) tv = __uint_as_float(v[i]);
                        p.target_logit[row] = tv;
                    }
                } else {
                    // (kEpiGate that keeps g and u: three buffers)
                    if (!TC_CHECK(holds(sC, staging_all, buf0, two_bufs ? 8192u : EPI == kEpiGate && p.keep ? 12288u : 4096u),
                                  kSiteSmemBounds)) {
                        failed = true;
                        break;
                    }
                    if constexpr (kLoads) {
                        if (loads) {
                            if (!warp_wait(aux_bar(ew, n_chunk & 1), (n_chunk >> 1) & 1, abort_flag, p.wait_limit, kSiteAuxLoad,
                                           lane)) {
                                failed = true;
                                break;
                            }
                            pending = false;
                        }
                    }
                    // without loads: the stores issued from these buffers have read them
                    if (!loads) {
                        if (lane == 0) wait_stores();
                        __syncwarp();
                    }
                    if constexpr (EPI == kEpiStore || EPI == kEpiStoreF32) {
                        constexpr int C = L::kChunk;
                        if (p.bias != nullptr) {
#pragma unroll
                            for (int i = 0; i < C / 32; ++i) {
                                const int col = x + i * 32 + lane;
                                st_shared_b16(sbias + (uint32_t)((i * 32 + lane) * 2),
                                              col < p.N ? static_cast<const unsigned short*>(p.bias)[col] : 0);
                            }
                            __syncwarp();
                        }
                        float f[C];
                        if constexpr (SPLIT) {
#pragma unroll
                            for (int i = 0; i < C; ++i) f[i] = 0.0f;
#pragma unroll 1
                            for (int r = 0; r < p.split; ++r) {
                                const uint32_t from = ptx::mapa(sA + (uint32_t)((c * 16 * 128 + q * 32 + lane) * 16),
                                                                2 * (uint32_t)r + rank);
#pragma unroll
                                for (int g = 0; g < C / 4; ++g) {
                                    uint32_t w[4];
                                    ptx::ld_cluster_v4(from + (uint32_t)(g * 2048), w[0], w[1], w[2], w[3]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) f[4 * g + e] += __uint_as_float(w[e]);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < C; ++i) f[i] *= alpha;
                        } else {
                            uint32_t v[C];
                            ptx::tmem_ld_32x32b_x32(trow + c * C, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                            if constexpr (C == 64)
                                ptx::tmem_ld_32x32b_x32(trow + c * C + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[C - 32]));
                            ptx::tmem_ld_wait();
                            if (c == c1 - 1) hand_back();
#pragma unroll
                            for (int i = 0; i < C; ++i) f[i] = __uint_as_float(v[i]) * alpha;
                        }
                        if (p.bias != nullptr) {
#pragma unroll
                            for (int i = 0; i < C; i += 8) {
                                uint32_t w[4];
                                ptx::ld_shared_v4(sbias + (uint32_t)(i * 2), w[0], w[1], w[2], w[3]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 b = unpack2<DT>(w[e]);
                                    f[i + 2 * e] += b.x;
                                    f[i + 2 * e + 1] += b.y;
                                }
                            }
                        }
                        if constexpr (EPI == kEpiStore) {
                            if (p.keep) {
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    ptx::st_shared_v4(swz(buf1, lane, j), pack2<DT>(f[8 * j], f[8 * j + 1]),
                                                      pack2<DT>(f[8 * j + 2], f[8 * j + 3]),
                                                      pack2<DT>(f[8 * j + 4], f[8 * j + 5]),
                                                      pack2<DT>(f[8 * j + 6], f[8 * j + 7]));
                            }
                            if (p.act != kActNone)
                                with_act(p.act, [&](auto tag) {
                                constexpr int ACT = decltype(tag)::value;
#pragma unroll
                                    for (int i = 0; i < C; i += 2) {
                                        const float2 o = parts(act_value2<ACT>(f2(f[i], f[i + 1])));
                                        f[i] = o.x, f[i + 1] = o.y;
                                    }
                                });
                            if (p.addend == 1) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    uint32_t w[4];
                                    ptx::ld_shared_v4(swz(buf0, lane, j), w[0], w[1], w[2], w[3]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float2 r = unpack2<DT>(w[e]);
                                        f[8 * j + 2 * e] += r.x;
                                        f[8 * j + 2 * e + 1] += r.y;
                                    }
                                }
                            } else if (p.addend == 2) {
                                // both buffers are read before the first is written
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    float r0, r1, r2, r3;
                                    ld_shared_f4(swz(j < 8 ? buf0 : buf1, lane, j & 7), r0, r1, r2, r3);
                                    f[4 * j] += r0;
                                    f[4 * j + 1] += r1;
                                    f[4 * j + 2] += r2;
                                    f[4 * j + 3] += r3;
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                ptx::st_shared_v4(swz(buf0, lane, j), pack2<DT>(f[8 * j], f[8 * j + 1]),
                                                  pack2<DT>(f[8 * j + 2], f[8 * j + 3]),
                                                  pack2<DT>(f[8 * j + 4], f[8 * j + 5]),
                                                  pack2<DT>(f[8 * j + 6], f[8 * j + 7]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (p.addend != 0) {
                                    float r0, r1, r2, r3;
                                    ld_shared_f4(swz(buf0, lane, j), r0, r1, r2, r3);
                                    f[4 * j] += r0;
                                    f[4 * j + 1] += r1;
                                    f[4 * j + 2] += r2;
                                    f[4 * j + 3] += r3;
                                }
                                ptx::st_shared_v4(swz(buf0, lane, j), __float_as_uint(f[4 * j]),
                                                  __float_as_uint(f[4 * j + 1]), __float_as_uint(f[4 * j + 2]),
                                                  __float_as_uint(f[4 * j + 3]));
                            }
                        }
                    } else if constexpr (EPI == kEpiGate) {
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            uint32_t g[32], u[32];
                            ptx::tmem_ld_32x32b_x32(trow + c * 64 + part * 32, g);
                            ptx::tmem_ld_32x32b_x32(trow + kHalf + c * 64 + part * 32, u);
                            ptx::tmem_ld_wait();
                            if (c == c1 - 1 && part == 1) hand_back();
                            if (p.keep) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    auto at = [&](const uint32_t(&r)[32], int i) { return __uint_as_float(r[8 * j + i]); };
                                    ptx::st_shared_v4(swz(buf0 + 4096, lane, part * 4 + j), pack2<DT>(at(g, 0), at(g, 1)),
                                                      pack2<DT>(at(g, 2), at(g, 3)), pack2<DT>(at(g, 4), at(g, 5)),
                                                      pack2<DT>(at(g, 6), at(g, 7)));
                                    ptx::st_shared_v4(swz(buf0 + 8192, lane, part * 4 + j), pack2<DT>(at(u, 0), at(u, 1)),
                                                      pack2<DT>(at(u, 2), at(u, 3)), pack2<DT>(at(u, 4), at(u, 5)),
                                                      pack2<DT>(at(u, 6), at(u, 7)));
                                }
                            }
                            float h[32];
                            with_act(p.act, [&](auto tag) {
                                constexpr int ACT = decltype(tag)::value;
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    const float2 o = parts(act_value2<ACT>(f2(__uint_as_float(g[i]), __uint_as_float(g[i + 1]))));
                                    h[i] = o.x * __uint_as_float(u[i]);
                                    h[i + 1] = o.y * __uint_as_float(u[i + 1]);
                                }
                            });
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                ptx::st_shared_v4(swz(buf0, lane, part * 4 + j), pack2<DT>(h[8 * j], h[8 * j + 1]),
                                                  pack2<DT>(h[8 * j + 2], h[8 * j + 3]),
                                                  pack2<DT>(h[8 * j + 4], h[8 * j + 5]),
                                                  pack2<DT>(h[8 * j + 6], h[8 * j + 7]));
                        }
                    } else if constexpr (EPI == kEpiGateGrad) {
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            uint32_t v[32];
                            ptx::tmem_ld_32x32b_x32(trow + c * 64 + part * 32, v);
                            ptx::tmem_ld_wait();
                            if (c == c1 - 1 && part == 1) hand_back();
                            with_act(p.act, [&](auto tag) {
                                constexpr int ACT = decltype(tag)::value;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    // this lane's row of g and u, replaced by dg and du
                                    uint32_t g[4], u[4];
                                    const uint32_t ag = swz(buf0, lane, part * 4 + j), au = ag + 4096;
                                    ptx::ld_shared_v4(ag, g[0], g[1], g[2], g[3]);
                                    ptx::ld_shared_v4(au, u[0], u[1], u[2], u[3]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float2 gf = unpack2<DT>(g[e]), uf = unpack2<DT>(u[e]);
                                        const float d0 = __uint_as_float(v[8 * j + 2 * e]);
                                        const float d1 = __uint_as_float(v[8 * j + 2 * e + 1]);
                                        g[e] = pack2<DT>(d0 * uf.x * act_slope<ACT>(gf.x), d1 * uf.y * act_slope<ACT>(gf.y));
                                        u[e] = pack2<DT>(d0 * act_value<ACT>(gf.x), d1 * act_value<ACT>(gf.y));
                                    }
                                    ptx::st_shared_v4(ag, g[0], g[1], g[2], g[3]);
                                    ptx::st_shared_v4(au, u[0], u[1], u[2], u[3]);
                                }
                            });
                        }
                    } else {  // kEpiLossGrad
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            uint32_t v[32];
                            ptx::tmem_ld_32x32b_x32(trow + c * 64 + part * 32, v);
                            ptx::tmem_ld_wait();
                            if (c == c1 - 1 && part == 1) hand_back();
                            const int rel = tcol - x - part * 32;
                            float f[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                f[i] = ex2_approx((__uint_as_float(v[i]) - lse) * 1.4426950408889634f);
                                if (i == rel) f[i] -= 1.0f;
                            }
                            // a row of weight 0 is 0 whatever its logits hold
                            auto put = [&](uint32_t to, float by) {
                                auto at = [&](int i) { return by == 0.0f ? 0.0f : f[i] * by; };
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    ptx::st_shared_v4(swz(to, lane, part * 4 + j), pack2<DT>(at(8 * j), at(8 * j + 1)),
                                                      pack2<DT>(at(8 * j + 2), at(8 * j + 3)),
                                                      pack2<DT>(at(8 * j + 4), at(8 * j + 5)),
                                                      pack2<DT>(at(8 * j + 6), at(8 * j + 7)));
                            };
                            put(buf0, scale);
                            if (p.keep) put(buf1, scale2);
                        }
                    }
                    constexpr bool kTail = EPI == kEpiStore || EPI == kEpiGate;
                    const int n8 = kTail ? p.N & ~7 : p.N;  // columns the tensor maps hold
                    if constexpr (kTail) {
                        if (n8 < p.N && n8 < x + L::kChunk && row < p.M) {
                            auto tail = [&](uint32_t buf, int o) {
                                store_tail(swz(buf, lane, (n8 - x) >> 3), p.tail_out[o], row * p.tail_ld[o] + n8, p.N - n8);
                            };
                            tail(buf0, 0);
                            if (EPI == kEpiStore && p.keep) tail(buf1, 1);
                            if (EPI == kEpiGate && p.keep) {
                                tail(buf0 + 4096, 1);
                                tail(buf0 + 8192, 2);
                            }
                        }
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (x < n8) {
                            ptx::tma_store_2d(&tm.out[0], buf0, x, row0);
                            if (EPI == kEpiGateGrad || ((EPI == kEpiStore || EPI == kEpiLossGrad) && p.keep))
                                ptx::tma_store_2d(&tm.out[1], buf1, x, row0);
                            if (EPI == kEpiGate && p.keep) {
                                ptx::tma_store_2d(&tm.out[1], buf0 + 4096, x, row0);
                                ptx::tma_store_2d(&tm.out[2], buf0 + 8192, x, row0);
                            }
                        }
                        ptx::bulk_commit_group();
                    }
                    if constexpr (kLoads) {
                        if (loads) {
                            // the next chunk's loads, into buffers whose stores have been read
                            int nx = x + L::kChunk, nrow = row0;
                            bool more = c + 1 < c1;
                            if (!more && !last_tile) {
                                int mb2, nb2;
                                layer_tile_coords(t + clusters, p, mb2, nb2);
                                nrow = mb2 * 256 + (int)rank * 128 + q * 32;
                                nx = nb2 * L::kOutN + c0 * L::kChunk;
                                more = nrow < p.M && c0 < chunk_end(nb2);
                            }
                            if (more) {
                                if (lane == 0) {
                                    wait_stores();
                                    issue_loads(nrow, nx, n_chunk + 1);
                                }
                                pending = true;
                            }
                        }
                    }
                    ++n_chunk;
                }
            }
            if (failed) break;
        }
        if (lane == 0) {
            // after an abort: loads under way land before shared memory goes away
            if (pending) wait_drain(aux_bar(ew, n_chunk & 1), (n_chunk >> 1) & 1, p.wait_limit);
            ptx::bulk_wait_group_read<0>();
        }
        __syncwarp();
    }

    if constexpr (SPLIT) {
        // the cluster's barrier before the partials are read takes every thread once:
        // the warps without an epilogue, and epilogue warps that gave up a wait
        if (!split_met) {
            __syncwarp();
            ptx::cluster_arrive();
            ptx::cluster_wait();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    // neither CTA leaves while the other may still signal into it
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, L::kTmemCols);
    }
}

}  // namespace tcgemm
