// The linear layer on microscaled operands: y = act(x w^T + bias) + residual on the
// tensor core's block-scaled products (tcgen05.mma, kind::mxf4 and kind::mxf8f6f4),
// which multiply the values of 32 of K by both operands' scales on the way into the
// fp32 accumulator.
//
// Both formats share one layout: a K step is 128 bytes of each row (256 values of
// e2m1, 128 of e4m3), one row of the 128-byte swizzle, and four products of 32 bytes.
// The scales of 128 rows by 4 blocks are one 512-byte tile in memory, in shared memory
// and, copied by tcgen05.cp, four columns of Tensor Memory: lane row % 32, column
// row / 32, byte block % 4, repeated for each quarter of the lanes.  A product names
// the byte it starts from in its instruction descriptor.
//
// Two kernels, chosen by estimated time (mx_ops.cuh):
//   pairs of CTAs on 256 x 256 tiles, persistent, the epilogue of one tile under the
//   products of the next.  Bound by the operands' way into the SM and, repeated, by power:
//   a step's 34 or 36 KB take 590 or 620 cycles at some 58 bytes a cycle, its products 512
//   (twice the products a step: 1,017); the next tile's wait for the columns that two
//   accumulators share adds some 800 a tile.
//   4096 x 4096 x 14336 81 us in 4 bits (6.0 PFLOP/s), 153 in 8 (3.1; the library's product
//   of the same operands 141); 4096 x 16384 x 4096 89 and 184; 4096 x 1024 x 8192 19 and 30.
//   For few tokens 128 weight rows by up to 128 tokens (the weights as the MMA's M), split
//   along K over a cluster.  Bound by HBM while it streams: one token, 4096 x 14336 7.9 us in
//   4 bits (31 MB: 4.6 at the copy rate), 12.8 in 8; 4096 x 4096 5.3 and 6.5.  3.5 us are a
//   launch's fixed path, as in layer_skinny_kernel.cuh.
#pragma once

#include "layer_skinny_kernel.cuh"
#include "mx_common.cuh"

namespace tcgemm {

namespace ptx {

// The tensor core's instructions take their operands from uniform registers.  A thread by
// itself pays for every one that it computed (110 to 150 cycles a product with scales, whose
// arithmetic takes 128), so here the whole warp walks the loop, on values and votes that are
// the same in every lane, and only the instructions are one lane's (4096 x 16384 x 4096, 4
// bits: 183 -> 91 us).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  elect.sync _|p, 0xffffffff;\n"
        "  selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(p));
    return p;
}

#define TC_MX_MMA(GROUP, KIND)                                                                              \
    asm volatile(                                                                                           \
        "{\n"                                                                                               \
        "  .reg .pred p, e;\n"                                                                              \
        "  setp.ne.b32 p, %4, 0;\n"                                                                         \
        "  setp.ne.b32 e, %7, 0;\n"                                                                         \
        "  @e tcgen05.mma.cta_group::" GROUP "." KIND " [%0], %1, %2, %3, [%5], [%6], p;\n"                \
        "}\n" ::"r"(d_tmem),                                                                                \
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(a_scale), "r"(b_scale), "r"(elected)     \
        : "memory")

// D (+)= A B with scales from Tensor Memory, on one CTA or a pair (GROUP); FMT as MxFormat.
template <int FMT, int GROUP>
__device__ __forceinline__ void mma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t a_scale,
                                       uint32_t b_scale, uint32_t accumulate, uint32_t elected) {
    if constexpr (FMT == kE2M1 && GROUP == 1) TC_MX_MMA("1", "kind::mxf4.block_scale.scale_vec::2X");
    if constexpr (FMT == kE2M1 && GROUP == 2) TC_MX_MMA("2", "kind::mxf4.block_scale.scale_vec::2X");
    if constexpr (FMT == kE4M3 && GROUP == 1) TC_MX_MMA("1", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    if constexpr (FMT == kE4M3 && GROUP == 2) TC_MX_MMA("2", "kind::mxf8f6f4.block_scale.scale_vec::1X");
}
#undef TC_MX_MMA

// One tile of scales, 32 rows of 16 bytes, into four columns of each quarter of the lanes
// (the pair's form: in both CTAs, each from its own shared memory).
template <int GROUP>
__device__ __forceinline__ void tmem_cp_scales(uint32_t tmem, uint64_t desc, uint32_t elected) {
    if constexpr (GROUP == 1)
        asm volatile("{\n  .reg .pred e;\n  setp.ne.b32 e, %2, 0;\n  @e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(tmem),
                     "l"(desc), "r"(elected)
                     : "memory");
    else
        asm volatile("{\n  .reg .pred e;\n  setp.ne.b32 e, %2, 0;\n  @e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(tmem),
                     "l"(desc), "r"(elected)
                     : "memory");
}

// `bytes` side by side, a multiple of 16, into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

// An arrival on an mbarrier of another CTA that hands over no memory, only Tensor Memory that
// has been read.  It releases nothing: that the next tile's products come after the reads
// rests on tcgen05.wait::ld, behind which the values are in registers, and on the fences of
// tcgen05 before this arrival and behind the wait for it.  With release at cluster scope it
// waited for whatever the SM had under way, 900 to 3,700 cycles, while the next tile waited
// for it.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// One word of another CTA's shared memory (addresses from mapa).
__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
}
// Counts `bytes` as landed that no copy will bring.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// mma_commit and its pair forms (to the leader alone, or to both CTAs).
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t elected) {
    asm volatile(
        "{\n  .reg .pred e;\n  setp.ne.b32 e, %1, 0;\n"
        "  @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"(elected)
        : "memory");
}
__device__ __forceinline__ void commit_both(uint32_t bar, uint32_t elected) {
    asm volatile(
        "{\n  .reg .pred e;\n  setp.ne.b32 e, %2, 0;\n"
        "  @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(bar),
        "h"((uint16_t)3), "r"(elected)
        : "memory");
}

}  // namespace ptx

constexpr int kMxStepBytes = 128;  // of each row a K step
__host__ __device__ constexpr int mx_step_blocks(int fmt) { return kMxStepBytes / mx_block_bytes(fmt); }  // 4 or 8
__host__ __device__ constexpr int mx_step_tiles(int fmt) { return mx_step_blocks(fmt) / 4; }              // scale tiles of 128 rows

// Instruction descriptor of a block-scaled product: both operands of the format, K-major,
// scales in powers of two; `a_byte`, `b_byte`: which byte of the scales' words is the first
// of this product's.
template <int FMT>
__host__ __device__ constexpr uint32_t mx_idesc(int m, int n, int a_byte, int b_byte) {
    const uint32_t type = FMT == kE2M1 ? 1u : 0u;
    return ((uint32_t)b_byte << 4) | (type << 7) | (type << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24) |
           ((uint32_t)a_byte << 29);
}

// Shared-memory descriptor of one tile of scales: no swizzle, groups of 8 rows of 16
// bytes 128 bytes apart.
__device__ __forceinline__ uint64_t mx_scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

// wait_bounded by a whole warp: every lane asks, and all go the same way.
__device__ __forceinline__ bool wait_uniform(uint32_t bar, uint32_t parity, volatile int* abort_flag, long long limit, unsigned site) {
    auto probe = [&]() {
        return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)) != 0;
    };
    if (probe()) return true;
    const long long t0 = clock64();
    while (!probe()) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
        if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
            *abort_flag = 1;
            record_timeout(site);
            return false;
        }
    }
    return true;
}

struct MxMaps {
    CUtensorMap x, w, xs, ws;
    CUtensorMap y, residual;  // pairs only
};

struct MxEpilogue {
    int act;
    const void *bias, *residual;
    void* y;
    long long ldr, ldy;
};

// ---- few tokens ----------------------------------------------------------------------------

constexpr int kMxSkinnySlots = 12;

struct MxSkinnyMaps {
    CUtensorMap x, w;
};

struct MxSkinnyParams {
    int T, N, nt, t_tiles;
    int blocks, k_steps;      // of 32 values; of 128 bytes
    int split, slots, stage_bytes, tmem_cols, scale_col;
    const uint8_t *xs, *ws;   // scales (copied plainly: a tensor map costs the host 0.4 us)
    int k_tiles;
    MxEpilogue e;
    long long wait_limit;
    int inject;
};

// Bias, activation and residual on four neighbouring columns of token t, stored.
template <int DT>
__device__ __forceinline__ void mx_finish4(const MxEpilogue& e, long long t, int n, int left, float (&o)[4]) {
    if (e.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) o[i] += load1<DT>(e.bias, n + i);
    }
    if (e.act != kActNone)
        with_act(e.act, [&](auto tag) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = act_value<decltype(tag)::value>(o[i]);
        });
    if (e.residual != nullptr) {
        float r[4];
        load4<DT>(e.residual, t * e.ldr + n, left, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += r[i];
    }
    store4<DT>(e.y, t * e.ldy + n, left, o);
}

template <int FMT, int DT>
__global__ void __launch_bounds__(kThreads) mx_skinny_kernel(const __grid_constant__ MxSkinnyMaps tm, const MxSkinnyParams p) {
    constexpr int kTiles = mx_step_tiles(FMT);           // scale tiles of a step
    constexpr int kScaleCols = 8 * kTiles;               // Tensor Memory columns of a step's scales, both operands
    constexpr uint32_t kScaleBytes = 512 * kTiles;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;
    const int S = p.slots;
    const uint32_t bar0 = ring + (uint32_t)(S * p.stage_bytes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (bar0 - raw) + 8 * (2 * kMxSkinnySlots + 1));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
#ifdef TCGEMM_CHECK
    if (bar0 + 8u * (2 * kMxSkinnySlots + 1) + 8u > raw + ptx::dynamic_smem_size() || p.nt * 512 > S * p.stage_bytes ||
        p.scale_col + 2 * kScaleCols > p.tmem_cols || p.nt > p.scale_col) {
        if (threadIdx.x == 0) record_timeout(kSiteSmemBounds);
        return;  // every CTA decides alike
    }
#endif
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMxSkinnySlots + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * kMxSkinnySlots);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int CS = p.split;
    const int rank = (int)blockIdx.x % CS;
    const int tile = (int)blockIdx.x / CS;
    const int n_tile = tile / p.t_tiles, t_tile = tile % p.t_tiles;
    const int n0 = n_tile * 128, t0 = t_tile * p.nt;
    const int tokens = min(p.nt, p.T - t0);
    const int own0 = tokens * rank / CS, own1 = tokens * (rank + 1) / CS;
    const int k0 = (int)((long long)p.k_steps * rank / CS), k1 = (int)((long long)p.k_steps * (rank + 1) / CS);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        ptx::mbar_init(done_bar, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm.w);
        ptx::prefetch_tmap(&tm.x);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr((const void*)tmem_slot), p.tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0 && p.inject == 0) {
            int stage = 0;
            uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
            ptx::grid_dependency_wait();
            // after the wait: whoever starts on this may take it that all kernels before this one are complete
            ptx::grid_launch_dependents();
            for (int kb = k0; kb < k1; ++kb) {
                if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.wait_limit, kSiteProducerEmpty)) break;
                const uint32_t dst = ring + (uint32_t)(stage * p.stage_bytes), fb = full_bar(stage);
                if (!TC_CHECK(holds(ring, (uint32_t)(S * p.stage_bytes), dst, (uint32_t)p.stage_bytes), kSiteSmemBounds)) break;
                // scale tiles of this step that exist
                const uint32_t here = 512u * (uint32_t)min(kTiles, p.k_tiles - kb * kTiles);
                ptx::mbar_arrive_expect_tx(fb, (uint32_t)((128 + p.nt) * kMxStepBytes) + 2 * here);
                const uint32_t xd = dst + 128 * kMxStepBytes, sd = xd + (uint32_t)(p.nt * kMxStepBytes);
                ptx::tma_load_2d(dst, &tm.w, fb, kb * kMxStepBytes, n0);
                ptx::bulk_load(sd, p.ws + ((long long)n_tile * p.k_tiles + kb * kTiles) * 512, here, fb);
                ptx::tma_load_2d(xd, &tm.x, fb, kb * kMxStepBytes, t0);
                ptx::bulk_load(sd + kScaleBytes, p.xs + ((long long)t_tile * p.k_tiles + kb * kTiles) * 512, here, fb);
                issued_mask |= 1u << stage;
                issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            for (int s = 0; s < S; ++s)
                if (issued_mask & (1u << s)) wait_drain(full_bar(s), (issued_phase >> s) & 1u, p.wait_limit);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (the whole warp) ----------------
        const uint32_t idesc = mx_idesc<FMT>(128, p.nt, 0, 0), elected = ptx::elect_one();
        int stage = 0, old_stage = 0;
        uint32_t phase = 0, old_phase = 0;
        for (int kb = k0; kb < k1; ++kb) {
            // two sets of scales in Tensor Memory: the products that read this one are complete
            if (kb - k0 >= 2) {
                if (!wait_uniform(empty_bar(old_stage), old_phase, abort_flag, p.wait_limit, kSiteMmaTmemEmpty)) break;
                if (++old_stage == S) {
                    old_stage = 0;
                    old_phase ^= 1u;
                }
            }
            if (!wait_uniform(full_bar(stage), phase, abort_flag, p.wait_limit, kSiteMmaFull)) break;
            ptx::tc_fence_after();
            const uint32_t src = ring + (uint32_t)(stage * p.stage_bytes);
            const uint32_t xsrc = src + 128 * kMxStepBytes, ssrc = xsrc + (uint32_t)(p.nt * kMxStepBytes);
            const uint32_t wcol = tmem + (uint32_t)(p.scale_col + ((kb - k0) & 1) * kScaleCols), xcol = wcol + 4 * kTiles;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                ptx::tmem_cp_scales<1>(wcol + 4 * i, mx_scale_desc(ssrc + 512 * i), elected);
                ptx::tmem_cp_scales<1>(xcol + 4 * i, mx_scale_desc(ssrc + kScaleBytes + 512 * i), elected);
            }
            const uint64_t wd = operand_desc<false>(src), xd = operand_desc<false>(xsrc);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int kPer = FMT == kE2M1 ? 2 : 1;  // blocks of a product
                if (kb * mx_step_blocks(FMT) + j * kPer < p.blocks) {
                    const uint32_t byte = (uint32_t)(j * kPer) & 3u, at = (uint32_t)(j * kPer) >> 2;
                    ptx::mma_mx<FMT, 1>(tmem, wd + 2 * j, xd + 2 * j, idesc | (byte << 4) | (byte << 29), wcol + 4 * at, xcol + 4 * at,
                                        ((kb - k0) | j) != 0, elected);
                }
            }
            ptx::commit_one(empty_bar(stage), elected);
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        ptx::commit_one(done_bar, elected);  // also after an abort: no MMA outlives the accumulator
        if (lane == 0) wait_drain(done_bar, 0, p.wait_limit);
        __syncwarp();
    } else {
        // ---------------- this CTA's partial out of TMEM ----------------
        const int q = warp & 3;
        ptx::grid_dependency_wait();
        if (warp_wait(done_bar, 0, abort_flag, 4 * p.wait_limit, kSiteEpilogueTmemFull, lane) && *abort_flag == 0) {
            ptx::tc_fence_after();
            const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
            const uint32_t col = (uint32_t)((q * 32 + lane) * 4);
            // the ring is idle: every load was consumed by an MMA, and every MMA is complete
#pragma unroll 1
            for (int c = 0; c < p.nt; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(trow + c, v);
                ptx::tmem_ld_wait();
                // [token][128 columns] fp32
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(ring + col + (uint32_t)((c + i) * 512)), "r"(v[i]) : "memory");
            }
        }
        ptx::tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, p.tmem_cols);
    }
    if (CS > 1) {
        __syncwarp();
        ptx::cluster_arrive();
        ptx::cluster_wait();
    }
    if (*abort_flag == 0) {
        // the previous kernel's reads and writes of what is read and written below are done
        ptx::grid_dependency_wait();
        // a warp on each of this CTA's tokens, a lane four columns, summed over the cluster first
        const int c = lane * 4, n = n0 + c, left = p.N - n;
        constexpr int kWarps = kThreads / 32;
        if (CS > 1) {
            if (CS <= 4)
                pull_sums<4, 4, 1>(ring, p.nt, CS, own0 + warp, own1, c);
            else
                pull_sums<8, 2, 1>(ring, p.nt, CS, own0 + warp, own1, c);
        }
        if (left > 0) {
#pragma unroll 1
            for (int tt = own0 + warp; tt < own1; tt += kWarps) {
                float o[4];
                ld_shared_f4(ring + (uint32_t)(tt * 512 + c * 4), o[0], o[1], o[2], o[3]);
                mx_finish4<DT>(p.e, t0 + tt, n, left, o);
            }
        }
    }
    if (CS > 1) {
        // no CTA leaves while another still reads its partial
        __syncwarp();
        ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    }
}

// ---- CTA pairs -----------------------------------------------------------------------------

template <int FMT>
struct MxPairLayout {
    static constexpr int kTiles = mx_step_tiles(FMT);
    static constexpr int kOperandBytes = 128 * kMxStepBytes;      // this CTA's 128 rows of x, or half of the tile's of w
    static constexpr int kScaleBytes = 512 * kTiles;              // 128 rows' scales of a step
    static constexpr int kStageBytes = 2 * kOperandBytes + 3 * kScaleBytes;  // x, w; scales of x's 128 rows and of all 256 of w
    static constexpr int kStride = (kStageBytes + 1023) / 1024 * 1024;
    static constexpr int kWarps = 8;     // epilogue: two for each 32 rows, on 128 columns each
    static constexpr int kThreads = 64 + 32 * kWarps;
    static constexpr int kSlots = 5;
    static constexpr int kStaging = 4096;  // an epilogue warp's 32 rows x 64 columns
    // full[8], empty[8], tmem_full[2], tmem_empty[2], shared, drain, residual[warps]
    static constexpr int kNumBars = 2 * kMaxStages + 6 + kWarps;
    // behind them: Tensor Memory's address, the abort flag, how far the warps came (MxCame)
    static constexpr int kWords = 32;
    static constexpr int kUsed = 1024 + kSlots * kStride + kWarps * kStaging + kNumBars * 8 + kWords;
    // All of an SM's shared memory, whatever is used of it, as the other kernels on pairs take
    // it: no other kernel's CTAs share the SM's bandwidth or its Tensor Memory with these.
    static constexpr int kSmem = 232448;
    static_assert(kSlots <= kMaxStages && kUsed <= kSmem, "shared memory");
    // Tensor Memory: the accumulators overlap in 128 columns, so that every stage of the ring
    // has a place of its own for its scales.  (With two places and 64 shared columns the
    // products of two steps ago had to be waited for: 4096 x 4096 x 14336, 4 bits, 88 us.)
    static constexpr int kScaleCols = 12 * kTiles;
    static constexpr int kSecond = 128;
    static constexpr int kScaleCol = kSecond + 256;
    static_assert(kScaleCol + kSlots * kScaleCols <= 512, "Tensor Memory");
};

// How far a CTA's warps came, for the way out after a wait that gave up.
enum MxCame { kCameLoads = 0, kCameSteps = 1, kCameTiles = 2 };  // stages loaded; committed (leader): stages, tiles

// After a wait that gave up in either CTA: whatever is still under way to this one lands, or a
// limit passes.  One thread of each CTA, between two barriers of the cluster; `loads0`, `loads1`:
// stages the two CTAs loaded; `steps`, `tiles`: what the leader committed.  Addresses: the first
// stage's barriers.
template <int S, int STAGE_BYTES>
__device__ __forceinline__ void mx_pair_settle(uint32_t rank, uint32_t full0, uint32_t empty0, uint32_t tfull0, uint32_t loads0,
                                               uint32_t loads1, uint32_t steps, uint32_t tiles, long long limit) {
    if (rank == 0) {
        // the leader's barrier counts both CTAs' bytes: a stage that only one of them loaded
        // (at most S: neither goes on before the products have read its last use) is made to
        // expect no more than that one's
        const uint32_t lo = min(loads0, loads1), hi = max(loads0, loads1);
        for (uint32_t k = lo; k < hi; ++k) {
            const uint32_t bar = full0 + 8u * (k % S);
            if (loads0 == lo)
                ptx::mbar_arrive_expect_tx(bar, STAGE_BYTES);
            else
                ptx::mbar_complete_tx(bar, STAGE_BYTES);
        }
        for (uint32_t k = hi > S ? hi - S : 0u; k < hi; ++k) wait_drain(full0 + 8u * (k % S), (k / S) & 1u, limit);
    }
    for (uint32_t k = steps > S ? steps - S : 0u; k < steps; ++k) wait_drain(empty0 + 8u * (k % S), (k / S) & 1u, limit);
    for (uint32_t t = tiles > 2u ? tiles - 2u : 0u; t < tiles; ++t) wait_drain(tfull0 + 8u * (t & 1u), (t >> 1) & 1u, limit);
}

struct MxPairParams {
    int M, N;
    int tiles_m, tiles_n;
    int blocks, k_steps;
    int raster_group;
    MxEpilogue e;
    long long wait_limit;
    int inject;
};

// Eight values of the bias, whose address is aligned to one.
template <int DT>
__device__ __forceinline__ uint4 bias8(const void* p, int n, int col, int cols) {
    if (((uintptr_t)p & 15) == 0) return load8<DT>(p, n, col, cols);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < cols) w[e >> 1] |= (uint32_t)static_cast<const unsigned short*>(p)[n + e] << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 64 neighbouring columns of a row, from x on, through the epilogue into the warp's 32-row
// staging buffer, where the residual is.
template <int DT>
__device__ __forceinline__ void mx_finish64(const MxEpilogue& e, int x, int left, uint32_t (&v)[2][32], uint32_t buf, int lane) {
    auto value = [&](int i) -> uint32_t& { return v[i >> 5][i & 31]; };
    if (e.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (8 * j >= left) break;
            float b[8];
            unpack8<DT>(bias8<DT>(e.bias, x + 8 * j, 8 * j, left), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) fadd_bits(value(8 * j + i), __float_as_uint(b[i]));
        }
    }
    if (e.act != kActNone)
        with_act(e.act, [&](auto tag) {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                const float2 o = parts(act_value2<decltype(tag)::value>(f2(__uint_as_float(value(i)), __uint_as_float(value(i + 1)))));
                value(i) = __float_as_uint(o.x);
                value(i + 1) = __float_as_uint(o.y);
            }
        });
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t at = swz(buf, lane, j);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(value(8 * j + i));
        if (e.residual != nullptr) {
            uint4 w;
            float r[8];
            ptx::ld_shared_v4(at, w.x, w.y, w.z, w.w);
            unpack8<DT>(w, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += r[i];
        }
        const uint4 o = pack8<DT>(f);
        ptx::st_shared_v4(at, o.x, o.y, o.z, o.w);
    }
}

template <int FMT, int DT>
__global__ void __launch_bounds__(MxPairLayout<FMT>::kThreads, 1)
    mx_pair_kernel(const __grid_constant__ MxMaps tm, const MxPairParams p) {
    using L = MxPairLayout<FMT>;
    constexpr int S = L::kSlots;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;
    const uint32_t staging = ring + S * L::kStride;
    const uint32_t bar0 = staging + L::kWarps * L::kStaging;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + (bar0 - raw) + 8 * L::kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* came = tmem_slot + 2;
    const uint32_t abort_at = bar0 + 8u * L::kNumBars + 4u, came_at = abort_at + 4u;
#ifdef TCGEMM_CHECK
    if (bar0 + 8u * L::kNumBars + L::kWords > raw + ptx::dynamic_smem_size()) {
        if (threadIdx.x == 0) record_timeout(kSiteSmemBounds);
        return;
    }
#endif
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * kMaxStages + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
    const uint32_t shared_bar = bar0 + 8u * (2 * kMaxStages + 4), drain_bar = shared_bar + 8u;
    auto residual_bar = [&](int w) { return drain_bar + 8u * (1 + w); };
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();  // 0 issues the MMAs

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(tfull_bar(a), 1);
            ptx::mbar_init(tempty_bar(a), 2 * L::kWarps);  // every epilogue warp of both CTAs
        }
        ptx::mbar_init(shared_bar, 2 * L::kWarps);
        ptx::mbar_init(drain_bar, 1);
        for (int w = 0; w < L::kWarps; ++w) ptx::mbar_init(residual_bar(w), 1);
        *abort_flag = 0;
        for (int i = 0; i < 3; ++i) came[i] = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm.x);
        ptx::prefetch_tmap(&tm.w);
        ptx::prefetch_tmap(&tm.xs);
        ptx::prefetch_tmap(&tm.ws);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr((const void*)tmem_slot), 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    const int tiles = p.tiles_m * p.tiles_n;
    auto coords = [&](int t, int& mb, int& nb) {  // groups of m-blocks, every second one backwards along n
        const int per_group = p.raster_group * p.tiles_n;
        const int grp = t / per_group, first_m = grp * p.raster_group;
        const int gm = min(p.tiles_m - first_m, p.raster_group);
        const int r = t - grp * per_group;
        mb = first_m + r % gm;
        nb = r / gm;
        if (grp & 1) nb = p.tiles_n - 1 - nb;
    };

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        if (lane == 0 && p.inject == 0) {
            int stage = 0;
            uint32_t phase = 0, loads = 0;
            bool ok = true;
            ptx::grid_dependency_wait();
            ptx::grid_launch_dependents();
            for (int t = pair; ok && t < tiles; t += pairs) {
                int mb, nb;
                coords(t, mb, nb);
                for (int kb = 0; kb < p.k_steps; ++kb) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.wait_limit, kSiteProducerEmpty)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = ring + stage * L::kStride;
                    if (!TC_CHECK(holds(ring, S * L::kStride, dst, L::kStageBytes), kSiteSmemBounds)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb_local = full_bar(stage);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(fb_local, 2 * L::kStageBytes);
                    const uint32_t fb = ptx::mapa(fb_local, 0), sd = dst + 2 * L::kOperandBytes;
                    const int kx = kb * kMxStepBytes, ks = kb * L::kTiles * 128;
                    ptx::tma_load_2d_pair(dst, &tm.x, fb, kx, mb * 256 + (int)rank * 128);
                    ptx::tma_load_2d_pair(dst + L::kOperandBytes, &tm.w, fb, kx, nb * 256 + (int)rank * 128);
                    ptx::tma_load_2d_pair(sd, &tm.xs, fb, ks, mb * 2 + (int)rank);
                    ptx::tma_load_2d_pair(sd + L::kScaleBytes, &tm.ws, fb, ks, nb * 2);
                    ptx::tma_load_2d_pair(sd + 2 * L::kScaleBytes, &tm.ws, fb, ks, nb * 2 + 1);
                    ++loads;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the last products' commits, to either CTA: nothing else waits for them
            for (int s = 0; ok && s < S; ++s) {
                ok = wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.wait_limit, kSiteProducerEmpty);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            came[kCameLoads] = loads;
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader only, the whole warp) ----------------
        if (rank == 0) {
            constexpr uint32_t idesc = mx_idesc<FMT>(256, 256, 0, 0);
            const uint32_t elected = ptx::elect_one();
            int stage = 0, tl = 0;
            uint32_t phase = 0, steps = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs, ++tl) {
                const int acc = tl & 1;
                // this accumulator's last tile is drained, and of the other's the columns they share
                if (!wait_uniform(tempty_bar(acc), ((tl >> 1) & 1) ^ 1u, abort_flag, p.wait_limit, kSiteMmaTmemEmpty) ||
                    !wait_uniform(shared_bar, (tl & 1) ^ 1u, abort_flag, p.wait_limit, kSiteMmaTmemEmpty)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem + (uint32_t)(acc * L::kSecond);
                for (int kb = 0; kb < p.k_steps; ++kb) {
                    // the stage was loaded once the products that read it before were complete,
                    // and its scales' place in Tensor Memory with it
                    if (!wait_uniform(full_bar(stage), phase, abort_flag, p.wait_limit, kSiteMmaFull)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t src = ring + stage * L::kStride, ssrc = src + 2 * L::kOperandBytes;
                    const uint32_t xcol = tmem + L::kScaleCol + (uint32_t)(stage * L::kScaleCols), wcol = xcol + 4 * L::kTiles;
#pragma unroll
                    for (int i = 0; i < L::kTiles; ++i) {
                        // w's 256 rows are eight neighbouring columns a tile of K
                        ptx::tmem_cp_scales<2>(xcol + 4 * i, mx_scale_desc(ssrc + 512 * i), elected);
                        ptx::tmem_cp_scales<2>(wcol + 8 * i, mx_scale_desc(ssrc + L::kScaleBytes + 512 * i), elected);
                        ptx::tmem_cp_scales<2>(wcol + 8 * i + 4, mx_scale_desc(ssrc + 2 * L::kScaleBytes + 512 * i), elected);
                    }
                    const uint64_t xd = operand_desc<false>(src), wd = operand_desc<false>(src + L::kOperandBytes);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        constexpr int kPer = FMT == kE2M1 ? 2 : 1;  // blocks of a product
                        if (kb * mx_step_blocks(FMT) + j * kPer < p.blocks) {
                            const uint32_t byte = (uint32_t)(j * kPer) & 3u, at = (uint32_t)(j * kPer) >> 2;
                            ptx::mma_mx<FMT, 2>(d_tmem, xd + 2 * j, wd + 2 * j, idesc | (byte << 4) | (byte << 29), xcol + 4 * at,
                                                wcol + 8 * at, (kb | j) != 0, elected);
                        }
                    }
                    ptx::commit_both(empty_bar(stage), elected);
                    ++steps;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                ptx::commit_both(tfull_bar(acc), elected);
            }
            __syncwarp();
            if (elected) {
                ptx::mma_commit_pair(drain_bar);
                wait_drain(drain_bar, 0, p.wait_limit);
                came[kCameSteps] = steps;
                came[kCameTiles] = (uint32_t)tl;  // (a tile that gave up is not counted)
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue (both CTAs): 32 rows x twice 64 columns a warp ----------------
        const int ew = warp - 2, q = warp & 3, half = ew >> 2;
        const uint32_t buf = staging + (uint32_t)(ew * L::kStaging), bar = residual_bar(ew);
        const int n8 = p.N & ~7;   // columns that y's tensor map holds (store_tail)
        ptx::grid_dependency_wait();
        ptx::grid_launch_dependents();
        bool pending = false;      // a load of the residual into buf is under way
        uint32_t loads = 0;        // and how many were before it
        int tl = 0;
        bool ok = TC_CHECK(holds(staging, L::kWarps * L::kStaging, buf, L::kStaging), kSiteSmemBounds);
        for (int t = pair; ok && t < tiles; t += pairs, ++tl) {
            int mb, nb;
            coords(t, mb, nb);
            const int acc = tl & 1;
            const int row0 = mb * 256 + (int)rank * 128 + q * 32;
            // 64 columns at a time; those that the accumulators share, the last 128 of the first
            // and the first of the second, before the others
            const int first = (acc ? 0 : 128) + half * 64;
            const int n0 = nb * 256;
            // the buffer is free once its last store has read it; then, where there is a
            // residual, its 32 x 64 values go there
            auto prepare = [&](int x) {
                if (row0 >= p.M || x >= p.N) return;
                if (lane == 0) {
                    ptx::bulk_wait_group_read<0>();
                    if (p.e.residual != nullptr) {
                        ptx::mbar_arrive_expect_tx(bar, L::kStaging);
                        ptx::tma_load_2d(buf, &tm.residual, bar, x, row0);
                    }
                }
                pending = p.e.residual != nullptr;
                __syncwarp();
            };
            prepare(n0 + first);
            if (!warp_wait(tfull_bar(acc), (tl >> 1) & 1, abort_flag, 4 * p.wait_limit, kSiteEpilogueTmemFull, lane)) break;
            ptx::tc_fence_after();
            const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * L::kSecond);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int c = i == 0 ? first : first ^ 128, x = n0 + c;
                if (i == 1) prepare(x);
                uint32_t v[2][32];
                ptx::tmem_ld_32x32b_x32(trow + c, v[0]);
                ptx::tmem_ld_32x32b_x32(trow + c + 32, v[1]);
                ptx::tmem_ld_wait();
                // handed back only where another tile waits for it: nothing else would hold the
                // leader until the arrival is there (see the way out)
                if ((i == 0 && t + pairs < tiles) || (i == 1 && t + 2 * pairs < tiles)) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa(i == 0 ? shared_bar : tempty_bar(acc), 0));
                }
                if (row0 >= p.M || x >= p.N) continue;
                if (pending) {
                    ok = warp_wait(bar, loads & 1, abort_flag, p.wait_limit, kSiteAuxLoad, lane);
                    if (!ok) break;
                    ++loads;
                    pending = false;
                }
                mx_finish64<DT>(p.e, x, p.N - x, v, buf, lane);
                if (n8 < p.N && n8 < x + 64 && row0 + lane < p.M)
                    store_tail(swz(buf, lane, (n8 - x) >> 3), p.e.y, (row0 + lane) * p.e.ldy + n8, p.N - n8);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && x < n8) {
                    ptx::tma_store_2d(&tm.y, buf, x, row0);
                    ptx::bulk_commit_group();
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            // after an abort: a load under way lands before shared memory goes away
            if (pending) wait_drain(bar, loads & 1, p.wait_limit);
            ptx::bulk_wait_group_read<0>();
        }
        __syncwarp();
    }
    ptx::tc_fence_before();
    __syncthreads();
    // The way out.  Neither CTA leaves while a signal or a copy of the other's may still be on its
    // way to it: what reaches the shared memory of a CTA that has left has no defined outcome,
    // its sender need not end, and no limit on a wait holds there.  This barrier alone does not
    // say so, since it orders nothing that was sent before it.  So each signal has its wait at
    // the receiver: the loads' barriers in the MMA warp, the commits of stages in either
    // producer, those of tiles in either epilogue, the accumulators' hand-backs in the MMA warp,
    // the last commit at drain_bar.  Where a wait gave up, the other CTA is told, and both make
    // up for what was not waited for.
    const bool gave_up = *abort_flag != 0;
    if (gave_up && threadIdx.x == 0) ptx::st_cluster_u32(ptx::mapa(abort_at, rank ^ 1u), 1u);
    if (gave_up)
        ptx::cluster_arrive();
    else
        ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
    if (*abort_flag != 0) {  // in both CTAs or in neither
        // this one's arrivals release: the hand-backs are there, and how far the warps came
        ptx::cluster_arrive();
        ptx::cluster_wait();
        if (threadIdx.x == 0) {
            const uint32_t lead = ptx::mapa(came_at, 0), other = ptx::mapa(came_at, 1);
            mx_pair_settle<S, L::kStageBytes>(rank, full_bar(0), empty_bar(0), tfull_bar(0), ptx::ld_cluster_u32(lead + 4 * kCameLoads),
                                              ptx::ld_cluster_u32(other + 4 * kCameLoads), ptx::ld_cluster_u32(lead + 4 * kCameSteps),
                                              ptx::ld_cluster_u32(lead + 4 * kCameTiles), p.wait_limit);
        }
        __syncwarp();
        ptx::cluster_arrive();
        ptx::cluster_wait();
    }
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace tcgemm
