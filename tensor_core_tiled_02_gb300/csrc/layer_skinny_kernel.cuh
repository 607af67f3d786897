// The layer operators' matrix product for few tokens: y = x w with x [T, K],
// where the time is that of streaming the weights once.
//
// The tile is computed transposed: the MMA's M is 128 weight columns and its N
// the tokens (rounded up to 16), so one token costs one sixteenth of a
// 256-row tile's products and none of the weights' bandwidth.  Weights come as
// [K, N] (the MMA's A operand MN-major) or [N, K] (K-major), as TMA loads them;
// x is the B operand, K-major.
//
// Memory-bound: what counts is enough bytes in flight on every SM.  N / 128
// column tiles alone rarely fill 152 SMs, so a thread-block cluster of up to 16
// CTAs shares each tile along K.  The fp32 partials then meet over distributed
// shared memory: each CTA of the cluster sums a share of the tile's tokens, in
// rank order (the same bits every time), a warp at a time on the 128 columns of
// one token, and applies the epilogue (layer_pair_kernel.cuh names them).
//   push  (a plain product of up to 4 tokens, up to 4 CTAs) every thread sends its
//         column's values straight from Tensor Memory to the CTA that sums the token,
//         which waits for the bytes on an mbarrier
//   pull  each CTA leaves its partial in its idle ring, the cluster meets at a
//         barrier, then reads
//
// One token, bf16: K = N = 4096 8.5 us (4.0 TB/s of weights), K = 4096, N = 14336 20.7
// (5.7 TB/s), K = N = 8192 22.7 (5.9 TB/s); gated block of 4096 x 14336, two launches,
// 57.2 (6.2 TB/s).
//
// Roles: warp 0 lane 0 loads, warp 1 lane 0 issues MMAs, warps 2-5 read the
// accumulator; all six reduce and store.  Every wait is bounded.
#pragma once

#include "layer_pair_kernel.cuh"

namespace tcgemm {

constexpr int kSkinnySlots = 12;     // most ring slots
constexpr int kSkinnySplit = 16;     // most CTAs sharing a tile (above 8 a non-portable cluster)
constexpr int kPushTokens = 4;       // most tokens whose partials are pushed, and most CTAs
constexpr int kPushSplit = 4;        // that push them to one another
constexpr int kSkinnyTileBytes = 128 * 64 * 2;  // one weight tile of one K step

struct SkinnyMaps {
    CUtensorMap w[2], x[2];
};

struct SkinnyParams {
    int T, N, nt;            // nt: tokens a tile, a multiple of 16: the MMA's N
    int t_tiles;             // ceil(T / nt)
    int k_steps, k_switch;   // 64-deep; steps >= k_switch read w[1], x[1] from their start (not kGate)
    int split, slots, stage_bytes, tmem_cols;
    int accs;                // kEpiLoss*: accumulators the K steps are dealt out to, summed in fp32
    int recv_bytes;          // PUSH: the buffer partials arrive in
    int weights_early;       // the previous kernel is this call's own and does not write the weights
    int act;
    const void* bias;
    const float* alpha;
    int alpha_rows;          // one alpha a token: [T]
    const void* addend;      // [T, N]: residual, or an fp32 running sum
    long long ld_addend;
    int addend_f32, out_f32;
    void* out;
    long long ld_out;
    void *keep0, *keep1;     // x w + bias; kEpiGate: g and u; kEpiGateGrad: du in keep1; kEpiLossGrad: with row_scale2
    long long ld_keep0, ld_keep1;
    const void *gate, *up;   // kEpiGateGrad: [T, N]
    long long ld_gate, ld_up;
    float2* stats;           // kEpiLossStats: [ceil(N / 128)][T]
    float* target_logit;
    const long long* target; // kEpiLoss*
    int col0;
    const float *lse, *row_scale, *row_scale2;
    long long wait_limit;
    int inject;
};

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Four bytes into another CTA's shared memory, counted on an mbarrier there.
__device__ __forceinline__ void st_async_b32(uint32_t cluster_addr, uint32_t v, uint32_t bar_cluster) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(cluster_addr), "r"(v),
                 "r"(bar_cluster)
                 : "memory");
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Four neighbouring values of a row, those from `left` on absent (0, not stored).
template <int DT>
__device__ __forceinline__ void load4(const void* p, long long at, int left, float (&f)[4]) {
    if (left >= 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(p) + at);
        const float2 a = unpack2<DT>(w.x), b = unpack2<DT>(w.y);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = i < left ? load1<DT>(p, at + i) : 0.0f;
    }
}

template <int DT>
__device__ __forceinline__ void store4(void* p, long long at, int left, const float (&f)[4]) {
    if (left >= 4) {
        *reinterpret_cast<uint2*>(static_cast<unsigned short*>(p) + at) =
            make_uint2(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) static_cast<unsigned short*>(p)[at + i] = pack1<DT>(f[i]);
    }
}

// Tokens tb, tb + 6, ... below tt_end of this warp: sums the cluster's partials of
// columns c .. c + 3 into this CTA's own, RANKS x BATCH reads under way at a time.
template <int RANKS, int BATCH, int TILES>
__device__ __forceinline__ void pull_sums(uint32_t ring, int nt, int ranks, int tb, int tt_end, int c) {
    constexpr int kWarps = kThreads / 32;
#pragma unroll 1
    for (; tb < tt_end; tb += kWarps * BATCH) {
#pragma unroll 1
        for (int i = 0; i < TILES; ++i) {
            float f[BATCH][4];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) f[u][0] = f[u][1] = f[u][2] = f[u][3] = 0.0f;
#pragma unroll 1
            for (int r0 = 0; r0 < ranks; r0 += RANKS) {
                uint32_t w[RANKS][BATCH][4];
#pragma unroll
                for (int r = 0; r < RANKS; ++r)
#pragma unroll
                    for (int u = 0; u < BATCH; ++u) {
                        const int tt = tb + u * kWarps;
                        w[r][u][0] = w[r][u][1] = w[r][u][2] = w[r][u][3] = 0u;
                        if (r0 + r < ranks && tt < tt_end)
                            ptx::ld_cluster_v4(ptx::mapa(ring, r0 + r) + (uint32_t)((i * nt + tt) * 512 + c * 4), w[r][u][0],
                                               w[r][u][1], w[r][u][2], w[r][u][3]);
                    }
#pragma unroll
                for (int r = 0; r < RANKS; ++r)
#pragma unroll
                    for (int u = 0; u < BATCH; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[u][e] += __uint_as_float(w[r][u][e]);
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int tt = tb + u * kWarps;
                if (tt < tt_end)
                    ptx::st_shared_v4(ring + (uint32_t)((i * nt + tt) * 512 + c * 4), __float_as_uint(f[u][0]),
                                      __float_as_uint(f[u][1]), __float_as_uint(f[u][2]), __float_as_uint(f[u][3]));
            }
        }
    }
}

template <bool WMN, int EPI, int DT, bool PUSH>
__global__ void __launch_bounds__(kThreads, 2)
    layer_skinny_kernel(const __grid_constant__ SkinnyMaps tm, const SkinnyParams p) {
    constexpr bool GATE = EPI == kEpiGate;
    constexpr bool LOSS = EPI == kEpiLossStats || EPI == kEpiLossGrad;  // logits, summed alike in both passes
    constexpr int kTiles = GATE ? 2 : 1;
    static_assert(!PUSH || EPI == kEpiStore, "pushed partials: one weight, the plain epilogue");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;
    const int S = p.slots;
    const uint32_t recv = ring + (uint32_t)(S * p.stage_bytes);
    const uint32_t bar0 = recv + (uint32_t)p.recv_bytes;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (bar0 - raw) + 8 * (2 * kSkinnySlots + 2));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
#ifdef TCGEMM_CHECK
    if (bar0 + 8u * (2 * kSkinnySlots + 2) + 8u > raw + ptx::dynamic_smem_size() ||
        (PUSH ? p.split * ((p.T + p.split - 1) / p.split) * 512 > p.recv_bytes || p.T > kPushTokens
                : kTiles * p.nt * 512 > S * p.stage_bytes)) {
        if (threadIdx.x == 0) record_timeout(kSiteSmemBounds);
        return;  // every CTA decides alike
    }
#endif
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kSkinnySlots + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * kSkinnySlots), recv_bar = done_bar + 8u;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int CS = p.split;
    const int rank = (int)blockIdx.x % CS;
    const int tile = (int)blockIdx.x / CS;
    const int n0 = (tile / p.t_tiles) * 128, t0 = (tile % p.t_tiles) * p.nt;
    // this CTA's tokens of the tile; pushed partials lie [rank][own token][128 columns]
    const int tokens = min(p.nt, p.T - t0);
    const int own0 = tokens * rank / CS, own1 = tokens * (rank + 1) / CS;
    const int most = (tokens + CS - 1) / CS;
    const int k0 = (int)((long long)p.k_steps * rank / CS), k1 = (int)((long long)p.k_steps * (rank + 1) / CS);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        ptx::mbar_init(done_bar, 1);
        ptx::mbar_init(recv_bar, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        if (PUSH && own1 > own0) ptx::mbar_arrive_expect_tx(recv_bar, (uint32_t)((own1 - own0) * CS * 512));
        ptx::prefetch_tmap(&tm.w[0]);
        ptx::prefetch_tmap(&tm.x[0]);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr((const void*)tmem_slot), p.tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (PUSH) {  // every CTA's mbarrier is ready before anyone sends to it
        ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    }
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0 && p.inject == 0) {
            int stage = 0;
            uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
            auto source = [&](int kb, int& k) {
                const int second = !GATE && kb >= p.k_switch;
                k = (second ? kb - p.k_switch : kb) * 64;
                return second;
            };
            auto load_weights = [&](int kb, int st) {
                if (!TC_CHECK(holds(ring, (uint32_t)(S * p.stage_bytes), ring + (uint32_t)(st * p.stage_bytes),
                                    (uint32_t)p.stage_bytes),
                              kSiteSmemBounds))
                    return;
                int k;
                const int second = source(kb, k);
                const uint32_t fb = full_bar(st);
                ptx::mbar_arrive_expect_tx(fb, (uint32_t)p.stage_bytes);
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const CUtensorMap* tw = &tm.w[GATE ? i : second];
                    const uint32_t d = ring + (uint32_t)(st * p.stage_bytes) + i * kSkinnyTileBytes;
                    if constexpr (WMN) {
                        ptx::tma_load_2d(d, tw, fb, n0, k);
                        ptx::tma_load_2d(d + kBoxBytes, tw, fb, n0 + 64, k);
                    } else {
                        ptx::tma_load_2d(d, tw, fb, k, n0);
                    }
                }
            };
            // Before the wait for the previous kernel, where that kernel is this call's own and
            // does not write the weights: the first of them.  (Elsewhere, asking L2 for them
            // before the wait measured slower: 8.7 -> 9.0 us for one step of one token at
            // K = N = 4096, 9.9 for four.)
            const int pre = p.weights_early ? min(S, k1 - k0) : 0;
            for (int i = 0; i < pre; ++i) load_weights(k0 + i, i);
            ptx::grid_dependency_wait();
            // after the wait: whoever starts on this may take it that all kernels before this one are complete
            ptx::grid_launch_dependents();
            for (int kb = k0; kb < k1; ++kb) {
                if (kb - k0 >= pre) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.wait_limit, kSiteProducerEmpty)) break;
                    load_weights(kb, stage);
                }
                int k;
                const int second = source(kb, k);
                ptx::tma_load_2d(ring + (uint32_t)(stage * p.stage_bytes + kTiles * kSkinnyTileBytes), &tm.x[second],
                                 full_bar(stage), k, t0);
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
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            const uint32_t idesc = layer_idesc(DT, WMN, false, 128, p.nt);
            int stage = 0;
            uint32_t phase = 0;
            // the loss's logits: consecutive runs of steps into accumulators of their own, as the
            // tensor core's accumulation truncates (layer_pair_kernel.cuh)
            const int run = LOSS ? (k1 - k0 + p.accs - 1) / p.accs : k1 - k0;
            uint32_t acc_tmem = tmem;
            int in_run = 0;
            for (int kb = k0; kb < k1; ++kb, ++in_run) {
                if (LOSS && in_run == run) {
                    in_run = 0;
                    acc_tmem += (uint32_t)p.nt;
                }
                if (!wait_bounded(full_bar(stage), phase, abort_flag, p.wait_limit, kSiteMmaFull)) break;
                ptx::tc_fence_after();
                const uint32_t src = ring + (uint32_t)(stage * p.stage_bytes);
                const uint64_t xd = operand_desc<false>(src + kTiles * kSkinnyTileBytes);
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const uint64_t wd = operand_desc<WMN>(src + i * kSkinnyTileBytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ptx::mma_f16_ss(acc_tmem + (uint32_t)(i * p.nt), wd + k * kSliceStep<WMN>,
                                        xd + k * kSliceStep<false>, idesc, (in_run | k) != 0);
                }
                ptx::mma_commit(empty_bar(stage));
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            ptx::mma_commit(done_bar);  // also after an abort: no MMA outlives the accumulator
            wait_drain(done_bar, 0, p.wait_limit);
        }
    } else {
        // ---------------- this CTA's partial out of TMEM ----------------
        const int q = warp & 3;
        // what the epilogue will read, towards this SM while the weights stream
        ptx::grid_dependency_wait();
        if constexpr (EPI == kEpiGateGrad) {
            const int n = n0 + q * 32;
            if (n < p.N)
                for (int t = own0 + lane; t < own1; t += 32) {
                    prefetch_l1(static_cast<const char*>(p.gate) + ((t0 + t) * p.ld_gate + n) * 2);
                    prefetch_l1(static_cast<const char*>(p.up) + ((t0 + t) * p.ld_up + n) * 2);
                }
            __syncwarp();
        }
        if constexpr (EPI == kEpiStore) {
            const int n = n0 + q * 32;  // 64 bytes of 16-bit values a warp
            if (lane == 0 && n < p.N) {
                if (p.bias != nullptr) prefetch_l1(static_cast<const char*>(p.bias) + (long long)n * 2);
                if (p.addend != nullptr)
                    for (int t = own0; t < own1; ++t)
                        prefetch_l1(static_cast<const char*>(p.addend) +
                                    ((long long)(t0 + t) * p.ld_addend + n) * (p.addend_f32 ? 4 : 2));
            }
            __syncwarp();
        }
        if (warp_wait(done_bar, 0, abort_flag, 4 * p.wait_limit, kSiteEpilogueTmemFull, lane) && *abort_flag == 0 &&
            TC_CHECK(kTiles * p.nt * (LOSS ? p.accs : 1) <= p.tmem_cols, kSiteTmemBounds)) {
            ptx::tc_fence_after();
            const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
            const uint32_t col = (uint32_t)((q * 32 + lane) * 4);
            // accumulators that hold anything (a short K range may leave the last ones empty)
            const int run = LOSS ? (k1 - k0 + p.accs - 1) / p.accs : 1;
            const int accs = LOSS ? (k1 - k0 + run - 1) / run : 1;
            auto load16 = [&](int c, uint32_t(&v)[16]) {
                tmem_ld_32x32b_x16(trow + c, v);
                if constexpr (LOSS) {
#pragma unroll 1
                    for (int a = 1; a < accs; ++a) {
                        uint32_t w[16];
                        tmem_ld_32x32b_x16(trow + a * p.nt + c, w);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) fadd_bits(v[i], w[i]);
                    }
                    if (accs > 1) return;
                }
                ptx::tmem_ld_wait();
            };
            (void)accs;
            if (PUSH) {
                uint32_t v[16];
                load16(0, v);
                // token t goes to the CTA whose share holds it
                int to = 0, first = 0, next = tokens / CS;
#pragma unroll
                for (int t = 0; t < kPushTokens; ++t) {
                    if (t < tokens) {
                        while (t >= next) {
                            ++to;
                            first = next;
                            next = tokens * (to + 1) / CS;
                        }
                        const uint32_t at = recv + (uint32_t)((rank * most + t - first) * 512) + col;
                        st_async_b32(ptx::mapa(at, to), v[t], ptx::mapa(recv_bar, to));
                    }
                }
            } else {
                // the ring is idle: every load was consumed by an MMA, and every MMA is complete
#pragma unroll 1
                for (int c = 0; c < kTiles * p.nt; c += 16) {
                    uint32_t v[16];
                    load16(c, v);
                    // [token][128 columns] fp32
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(ring + col + (uint32_t)((c + i) * 512)), "r"(v[i]) : "memory");
                }
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
    bool here = true;  // the partials of this CTA's tokens are within reach
    if (PUSH) {
        here = own1 == own0 || warp_wait<true>(recv_bar, 0, abort_flag, p.wait_limit, kSiteReduceData, lane);
    } else if (CS > 1) {
        __syncwarp();
        ptx::cluster_arrive();
        ptx::cluster_wait();
    }
    if (here && *abort_flag == 0) {
        // the previous kernel's reads and writes of what is read and written below are done
        ptx::grid_dependency_wait();
        const float one_alpha = p.alpha != nullptr && !p.alpha_rows ? *p.alpha : 1.0f;
        // A warp on each of this CTA's tokens, a lane four columns.  Where partials are
        // pulled, first the sums over the cluster, kept in this CTA's own partial (nobody
        // else reads these tokens of it): all ranks' values of a batch of tokens at once,
        // so that the reads of other CTAs' shared memory overlap.
        const int c = lane * 4, n = n0 + c, left = p.N - n;
        const int tt_begin = own0 + warp, tt_end = own1;
        constexpr int kWarps = kThreads / 32;
        if (CS > 1 && !PUSH) {
            if (CS <= 4)
                pull_sums<4, 4, kTiles>(ring, p.nt, CS, tt_begin, tt_end, c);
            else
                pull_sums<8, 2, kTiles>(ring, p.nt, CS, tt_begin, tt_end, c);
        }
#pragma unroll 1
        for (int tt = tt_begin; tt < tt_end; tt += kWarps) {
            const int t = t0 + tt;
            float f[kTiles][4];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                if (PUSH) {
                    f[i][0] = f[i][1] = f[i][2] = f[i][3] = 0.0f;
#pragma unroll 4
                    for (int r = 0; r < CS; ++r) {
                        float a, b, d, e;
                        ld_shared_f4(recv + (uint32_t)((r * most + tt - own0) * 512 + c * 4), a, b, d, e);
                        f[i][0] += a, f[i][1] += b, f[i][2] += d, f[i][3] += e;
                    }
                } else {
                    ld_shared_f4(ring + (uint32_t)((i * p.nt + tt) * 512 + c * 4), f[i][0], f[i][1], f[i][2], f[i][3]);
                }
            }
            float o[4];
            if constexpr (EPI == kEpiLossStats) {
                float m = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e >= left) f[0][e] = -INFINITY;  // columns from N on are no words
                    m = fmaxf(m, f[0][e]);
                }
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
                const float mf = m == -INFINITY ? 0.0f : m;
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += ex2_approx((f[0][e] - mf) * 1.4426950408889634f);
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
                if (lane == 0) p.stats[(size_t)(n0 >> 7) * p.T + t] = make_float2(m, sum);
                const long long rel = p.target[t] - n;
                if (rel >= 0 && rel < 4 && rel < left)
                    p.target_logit[t] = rel == 0 ? f[0][0] : rel == 1 ? f[0][1] : rel == 2 ? f[0][2] : f[0][3];
                __syncwarp();
                continue;
            }
            if (left <= 0) continue;
            if constexpr (EPI == kEpiLossGrad) {
                const float lse = p.lse[t], scale = p.row_scale[t];
                const long long rel = p.target[t] - p.col0 - n;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[0][e] = ex2_approx((f[0][e] - lse) * 1.4426950408889634f) - (rel == e ? 1.0f : 0.0f);
                    o[e] = scale == 0.0f ? 0.0f : f[0][e] * scale;
                }
                store4<DT>(p.out, t * p.ld_out + n, left, o);
                if (p.keep0 != nullptr) {
                    const float scale2 = p.row_scale2[t];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = scale2 == 0.0f ? 0.0f : f[0][e] * scale2;
                    store4<DT>(p.keep0, t * p.ld_keep0 + n, left, o);
                }
            } else if constexpr (EPI == kEpiGateGrad) {
                float g[4], u[4], du[4];
                load4<DT>(p.gate, t * p.ld_gate + n, left, g);
                load4<DT>(p.up, t * p.ld_up + n, left, u);
                with_act(p.act, [&](auto tag) {
                    constexpr int ACT = decltype(tag)::value;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[e] = f[0][e] * u[e] * act_slope<ACT>(g[e]);
                        du[e] = f[0][e] * act_value<ACT>(g[e]);
                    }
                });
                store4<DT>(p.out, t * p.ld_out + n, left, o);
                store4<DT>(p.keep1, t * p.ld_keep1 + n, left, du);
            } else if constexpr (GATE) {
                if (p.keep0 != nullptr) {
                    store4<DT>(p.keep0, t * p.ld_keep0 + n, left, f[0]);
                    store4<DT>(p.keep1, t * p.ld_keep1 + n, left, f[1]);
                }
                with_act(p.act, [&](auto tag) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = act_value<decltype(tag)::value>(f[0][e]) * f[1][e];
                });
                store4<DT>(p.out, t * p.ld_out + n, left, o);
            } else {
                const float alpha = p.alpha_rows ? p.alpha[t] : one_alpha;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = f[0][e] * alpha;
                    if (p.bias != nullptr && e < left) o[e] += load1<DT>(p.bias, n + e);
                }
                if (p.keep0 != nullptr) store4<DT>(p.keep0, t * p.ld_keep0 + n, left, o);
                if (p.act != kActNone)
                    with_act(p.act, [&](auto tag) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = act_value<decltype(tag)::value>(o[e]);
                    });
                if (p.addend != nullptr) {
                    if (p.addend_f32) {
                        const float* a = static_cast<const float*>(p.addend) + t * p.ld_addend + n;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (e < left) o[e] += a[e];
                    } else {
                        float a[4];
                        load4<DT>(p.addend, t * p.ld_addend + n, left, a);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] += a[e];
                    }
                }
                if (p.out_f32) {
                    float* d = static_cast<float*>(p.out) + t * p.ld_out + n;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) d[e] = o[e];
                } else {
                    store4<DT>(p.out, t * p.ld_out + n, left, o);
                }
            }
        }
    }
    if (CS > 1) {
        // no CTA leaves while another still reads its partial or sends to it
        __syncwarp();
        ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    }
}

}  // namespace tcgemm
