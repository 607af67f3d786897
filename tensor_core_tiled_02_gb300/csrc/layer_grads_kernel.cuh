// The products of one backward pass in one launch: dx and the weight gradients
// read the same factors and not one another, but run to very different lengths
// (dx has the layer's width as its K, a weight gradient the tokens).  One after
// the other, each ends on a partly filled wave of 256 x 256 pair tiles; together,
// the pairs that the last wave of long tiles leaves idle take short ones.
//
//   long group   tiles of the larger K, dealt out in rounds over the pairs; the
//                last round reaches only `rem` of them
//   short group  first `d` tiles each to the pairs without a tile in that round (as
//                many as one long tile lasts), then in rounds over all, these pairs first
//
// 2001 tokens, 2048 x 8192: dx 64 tiles of 128 steps and dw 256 tiles of 32 on 76
// pairs take 91 us one after the other, 75 together (1790 TFLOP/s; 73 at the measured
// peak); dx and the three weight gradients of the gated block, 4096 tokens, 4096 x 14336,
// 1255 us (1916 TFLOP/s, one launch).  Bound by the tensor pipe, 88 and 96 % of the
// cycles busy.
//
// Tiles, ring, roles and waits are layer_pair_kernel.cuh's, with the operands'
// major order a property of the problem; the epilogue is y = alpha v.
#pragma once

#include "layer_pair_kernel.cuh"

namespace tcgemm {

constexpr int kGradsProblems = 4;

struct GradsMaps {
    // the i-th problem's operands are a[i], b[i]; its second pair (K continued) a[4], b[4]
    CUtensorMap a[kGradsProblems + 1], b[kGradsProblems + 1];
    CUtensorMap out[kGradsProblems];
};

struct GradsProblem {
    int M, N, tiles_m, tiles_n;
    int k_steps, k_switch;  // steps >= k_switch read the second pair
    int a_mn, b_mn;         // operand stored [K, M] (or [K, N]) rather than [M, K] ([N, K])
    int alpha_rows;         // one alpha a row
    const float* alpha;     // device scalar or [M], NULL for 1
    void* out;              // the output again, for columns from N & ~7 on (store_tail)
    long long ld_out;
};

struct GradsParams {
    GradsProblem q[kGradsProblems];
    int longs;              // problems [0, longs) form the long group
    int tiles[2];           // of the long and the short group
    int rounds, rem, d;     // the long group's full rounds, the tiles of its last, and see above
    int raster_group;
    long long wait_limit;
    int inject;
};

// The i-th tile of pair c of P: problem and tile in it.  False when it has none.
__device__ __forceinline__ bool grads_tile(const GradsParams& p, int c, int P, int i, int& prob, int& mb, int& nb) {
    int group = 1, t;
    const int free_pairs = P - p.rem;
    if (i < p.rounds || (i == p.rounds && c < p.rem)) {
        group = 0;
        t = c + i * P;
    } else if (c < p.rem) {
        t = p.d * free_pairs + (i - p.rounds - 1) * P + free_pairs + c;
    } else {
        const int j = i - p.rounds;
        t = j < p.d ? c - p.rem + j * free_pairs : p.d * free_pairs + (j - p.d) * P + c - p.rem;
    }
    if (t >= p.tiles[group]) return false;
    prob = group == 0 ? 0 : p.longs;
    while (t >= p.q[prob].tiles_m * p.q[prob].tiles_n) {
        t -= p.q[prob].tiles_m * p.q[prob].tiles_n;
        ++prob;
    }
    const GradsProblem& q = p.q[prob];
    const int g = p.raster_group, per_group = g * q.tiles_n, grp = t / per_group, first_m = grp * g;
    const int gm = min(q.tiles_m - first_m, g), r = t - grp * per_group;
    mb = first_m + r % gm;
    nb = r / gm;
    if (grp & 1) nb = q.tiles_n - 1 - nb;
    return true;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
    layer_grads_kernel(const __grid_constant__ GradsMaps tm, const __grid_constant__ GradsParams p) {
    constexpr int kHalf = kTileN / 2;
    using L = LayerPairLayout<kEpiStore, false>;
    constexpr int S = L::kSlots;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    const uint32_t sA = base;
    const uint32_t sB = sA + S * L::kABytes;
    const uint32_t sC = sB + S * L::kBBytes;
    const uint32_t bar0 = sC + L::kWarps * L::kWarpStaging;
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
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(tfull_bar(a), 1);
            ptx::mbar_init(tempty_bar(a), 2 * L::kWarps);
        }
        ptx::mbar_init(drain_bar, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
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
    auto stage_ok = [&](int st) {
        const uint32_t bars = (uint32_t)L::kNumBars * 8u;
        return holds(bar0, bars, empty_bar(st), 8) && holds(bar0, bars, full_bar(st), 8) &&
               holds(sA, (uint32_t)(S * L::kABytes), sA + st * L::kABytes, L::kABytes) &&
               holds(sB, (uint32_t)(S * L::kBBytes), sB + st * L::kBBytes, L::kBBytes);
    };
    (void)stage_ok;
    const int pair = blockIdx.x >> 1;
    const int P = gridDim.x >> 1;

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        if (lane == 0 && p.inject == 0) {
            int stage = 0;
            uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
            bool ok = true;
            ptx::grid_dependency_wait();
            ptx::grid_launch_dependents();
            int prob, mb, nb;
            for (int i = 0; ok && grads_tile(p, pair, P, i, prob, mb, nb); ++i) {
                const GradsProblem& q = p.q[prob];
                const int m0 = mb * 256 + (int)rank * 128, n0 = nb * kTileN + (int)rank * kHalf;
                const int KB = q.k_steps, k_switch = q.k_switch, a_mn = q.a_mn, b_mn = q.b_mn;
                for (int kb = 0; kb < KB; ++kb) {
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
                    const uint32_t fb = ptx::mapa(fb_local, 0);
                    const bool second = kb >= k_switch;
                    const int k0 = (second ? kb - k_switch : kb) * 64;
                    const CUtensorMap* ta = &tm.a[second ? kGradsProblems : prob];
                    const CUtensorMap* tb = &tm.b[second ? kGradsProblems : prob];
                    const uint32_t a = sA + stage * L::kABytes, b = sB + stage * L::kBBytes;
                    if (a_mn) {
                        ptx::tma_load_2d_pair(a, ta, fb, m0, k0);
                        ptx::tma_load_2d_pair(a + kBoxBytes, ta, fb, m0 + 64, k0);
                    } else {
                        ptx::tma_load_2d_pair(a, ta, fb, k0, m0);
                    }
                    if (b_mn) {
                        ptx::tma_load_2d_pair(b, tb, fb, n0, k0);
                        ptx::tma_load_2d_pair(b + kBoxBytes, tb, fb, n0 + 64, k0);
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
            if (rank == 0)
                for (int s = 0; s < S; ++s)
                    if (issued_mask & (1u << s)) wait_drain(full_bar(s), (issued_phase >> s) & 1u, p.wait_limit);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader only) ----------------
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int prob, mb, nb;
            for (int i = 0; ok && grads_tile(p, pair, P, i, prob, mb, nb); ++i) {
                const GradsProblem& q = p.q[prob];
                const int acc = i & 1;
                if (!wait_bounded<true>(tempty_bar(acc), ((i >> 1) & 1) ^ 1u, abort_flag, p.wait_limit, kSiteMmaTmemEmpty)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kTileN);
                const uint32_t idesc = layer_idesc(DT, q.a_mn != 0, q.b_mn != 0, 256, kTileN);
                const uint64_t a_base = q.a_mn ? operand_desc<true>(0) : operand_desc<false>(0);
                const uint64_t b_base = q.b_mn ? operand_desc<true>(0) : operand_desc<false>(0);
                const uint32_t a_step = q.a_mn ? kSliceStep<true> : kSliceStep<false>;
                const uint32_t b_step = q.b_mn ? kSliceStep<true> : kSliceStep<false>;
                const int KB = q.k_steps;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!TC_CHECK(stage_ok(stage), kSiteSmemBounds)) {
                        ok = false;
                        break;
                    }
                    if (!wait_bounded(full_bar(stage), phase, abort_flag, p.wait_limit, kSiteMmaFull)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    // the start address goes into the descriptor's low field (16-byte units)
                    const uint64_t ad0 = a_base | ((sA + stage * L::kABytes) >> 4);
                    const uint64_t bd0 = b_base | ((sB + stage * L::kBBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ptx::mma_f16_ss_pair(d_tmem, ad0 + k * a_step, bd0 + k * b_step, idesc, kb | k);
                    ptx::mma_commit_pair_multicast(empty_bar(stage), 0x3);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                ptx::mma_commit_pair_multicast(tfull_bar(acc), 0x3);
            }
            ptx::mma_commit_pair(drain_bar);
            wait_drain(drain_bar, 0, p.wait_limit);
        }
    } else {
        // ---------------- epilogue (both CTAs): 32 rows x 256 columns a warp ----------------
        const int q4 = warp & 3;
        const uint32_t stg = sC + (uint32_t)((warp - 2) * L::kWarpStaging);
        const uint32_t lane_base = tmem_base + ((uint32_t)(q4 * 32) << 16);
        ptx::grid_dependency_wait();
        ptx::grid_launch_dependents();
        unsigned n_chunk = 0;
        int prob, mb, nb;
        for (int i = 0; grads_tile(p, pair, P, i, prob, mb, nb); ++i) {
            const GradsProblem& q = p.q[prob];
            const int acc = i & 1;
            const int row0 = mb * 256 + (int)rank * 128 + q4 * 32, n0 = nb * kTileN;
            const int chunks = row0 < q.M ? min(kTileN / 64, (q.N - n0 + 63) / 64) : 0;
            float alpha = 1.0f;
            if (q.alpha != nullptr) alpha = !q.alpha_rows ? *q.alpha : row0 + lane < q.M ? q.alpha[row0 + lane] : 0.0f;
            if (!warp_wait(tfull_bar(acc), (i >> 1) & 1, abort_flag, 4 * p.wait_limit, kSiteEpilogueTmemFull, lane)) break;
            ptx::tc_fence_after();
            const uint32_t trow = lane_base + (uint32_t)(acc * kTileN);
            int p2, m2, n2;
            const bool last = !grads_tile(p, pair, P, i + 1, p2, m2, n2);  // no MMA waits for its accumulator
            auto hand_back = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0 && !last) ptx::mbar_arrive_cluster(ptx::mapa(tempty_bar(acc), 0));
            };
            if (chunks == 0) hand_back();
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const uint32_t buf = stg + (n_chunk & 3) * 4096u;
                if (!TC_CHECK(holds(sC, (uint32_t)(L::kWarps * L::kWarpStaging), buf, 4096u) && acc * kTileN + kTileN <= L::kTmemCols,
                              kSiteSmemBounds))
                    break;
                if (lane == 0) ptx::bulk_wait_group_read<3>();
                __syncwarp();
                uint32_t v[64];
                ptx::tmem_ld_32x32b_x32(trow + c * 64, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                ptx::tmem_ld_32x32b_x32(trow + c * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                ptx::tmem_ld_wait();
                if (c == chunks - 1) hand_back();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    auto at = [&](int e) { return __uint_as_float(v[8 * j + e]) * alpha; };
                    ptx::st_shared_v4(swz(buf, lane, j), pack2<DT>(at(0), at(1)), pack2<DT>(at(2), at(3)),
                                      pack2<DT>(at(4), at(5)), pack2<DT>(at(6), at(7)));
                }
                const int x = n0 + c * 64, n8 = q.N & ~7;
                if (n8 < q.N && n8 < x + 64 && row0 + lane < q.M)
                    store_tail(swz(buf, lane, (n8 - x) >> 3), q.out, (row0 + lane) * q.ld_out + n8, q.N - n8);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (x < n8) ptx::tma_store_2d(&tm.out[prob], buf, x, row0);
                    ptx::bulk_commit_group();
                }
                ++n_chunk;
            }
        }
        if (lane == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
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
