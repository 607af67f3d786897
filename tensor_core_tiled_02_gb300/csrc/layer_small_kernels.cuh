// The layer operators' bandwidth-bound passes around their matrix products:
// the slope of a linear layer's activation with the bias gradient's column
// sums, and the reductions of the vocabulary cross entropy.  All sums are in
// fp32, in a fixed order: the same inputs give the same bits.
#pragma once

#include "layer_common.cuh"

namespace tcgemm {

// ---- linear layer: dpre = dy act'(pre), column sums of dpre ------------------------
//
// A block takes kSlopeRows rows x 256 columns: 32 groups of 8 columns (16
// bytes) x 8 rows at a time.  Reads dy and pre once, writes dpre once; the
// block's column sums (of the unrounded products) go to partial[row block][N].
// 2001 x 8192, bf16, GELU: 22 us from a cold cache, 4.6 TB/s of the 98 MB.
constexpr int kSlopeRows = 64;
constexpr int kSlopeCols = 256;

struct SlopeParams {
    const void* dy;
    const void* pre;   // NULL: no activation
    void* dpre;        // NULL: column sums only
    float* partial;    // NULL: no column sums
    long long ld_dy, ld_pre, ld_dpre;
    int rows, cols, act;
    int col_blocks;    // grid: row block * col_blocks + column block
};

template <int DT>
__global__ void __launch_bounds__(256, 5) layer_slope_kernel(const SlopeParams p) {
    __shared__ float sums[8][kSlopeCols];
    const int cg = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int cb = blockIdx.x % p.col_blocks, rb = blockIdx.x / p.col_blocks;
    const int col = cb * kSlopeCols + cg * 8;
    const int r0 = rb * kSlopeRows;
    const int r1 = min(p.rows, r0 + kSlopeRows);
    F2 acc[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (col < p.cols) {
        const bool whole = col + 8 <= p.cols;
        with_act(p.pre ? p.act : kActNone, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
            constexpr int U = 2;  // rows under way per thread
            if (whole) {
                for (int rb = r0 + rl; rb < r1; rb += 8 * U) {
                    uint4 w[U], z[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const long long r = rb + 8 * u;
                        if (r >= r1) continue;
                        w[u] = *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(p.dy) + r * p.ld_dy + col);
                        if constexpr (ACT != kActNone)
                            z[u] = *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(p.pre) + r * p.ld_pre + col);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const long long r = rb + 8 * u;
                        if (r >= r1) continue;
                        const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w}, zs[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
                        uint32_t os[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 d = unpack2<DT>(ws[e]);
                            F2 f = f2(d.x, d.y);
                            if constexpr (ACT != kActNone) {
                                const float2 g = unpack2<DT>(zs[e]);
                                f = mul2(f, act_slope2<ACT>(f2(g.x, g.y)));
                            }
                            acc[e] = add2(acc[e], f);
                            const float2 o = parts(f);
                            os[e] = pack2<DT>(o.x, o.y);
                        }
                        if (p.dpre)
                            *reinterpret_cast<uint4*>(static_cast<unsigned short*>(p.dpre) + r * p.ld_dpre + col) =
                                make_uint4(os[0], os[1], os[2], os[3]);
                    }
                }
            } else {
                for (long long r = r0 + rl; r < r1; r += 8)
                    for (int e = 0; e < 8 && col + e < p.cols; ++e) {
                        float d = load1<DT>(p.dy, r * p.ld_dy + col + e);
                        if constexpr (ACT != kActNone) d *= act_slope<ACT>(load1<DT>(p.pre, r * p.ld_pre + col + e));
                        if (p.dpre) static_cast<unsigned short*>(p.dpre)[r * p.ld_dpre + col + e] = pack1<DT>(d);
                        acc[e >> 1] = add2(acc[e >> 1], e & 1 ? f2(0.0f, d) : f2(d, 0.0f));
                    }
            }
        });
    }
    if (p.partial == nullptr) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = parts(acc[e]);
        sums[rl][cg * 8 + 2 * e] = a.x;
        sums[rl][cg * 8 + 2 * e + 1] = a.y;
    }
    __syncthreads();
    const int c = cb * kSlopeCols + threadIdx.x;
    if (c < p.cols) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
        p.partial[(size_t)rb * p.cols + c] = s;
    }
}

// dbias[c] = sum over row blocks of partial[b][c], rounded once.  32 columns a
// block, 8 slices of the row blocks side by side.
template <int DT>
__global__ void __launch_bounds__(256) layer_column_sum_kernel(const float* partial, void* out, int blocks, int cols) {
    __shared__ float sums[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float s = 0.0f;
    if (c < cols)
        for (int b = slice; b < blocks; b += 8) s += partial[(size_t)b * cols + c];
    sums[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0 && c < cols) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
        static_cast<unsigned short*>(out)[c] = pack1<DT>(s);
    }
}

// ---- vocabulary cross entropy --------------------------------------------------------

struct LossParams {
    const float2* stats;        // [parts][rows]
    const float* target_logit;  // [rows], set where the target is a word
    const long long* target;
    float* row_loss;            // [rows]
    float* lse;                 // [rows]
    int rows, parts;
    long long vocab, ignore_index;
    float* total;               // at most 32 rows (one block): their sum or mean too, else NULL
    int mean;
};

// lse = max + ln(sum over parts of s_i exp(m_i - max)); loss = lse - target's
// logit.  An ignored row's loss is 0; a target that is neither ignored nor a
// word makes its row's loss NaN.  32 rows a block, 32 slices of the parts, each
// slice four independent loads at a time: the pass is latency (1000 rows x 391
// parts, 3.2 MB, 10 us from a cold cache).
__global__ void __launch_bounds__(1024) layer_loss_rows_kernel(const LossParams p) {
    __shared__ float2 part[32][33];
    const int l = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int row = blockIdx.x * 32 + l;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float m = -INFINITY, s = 0.0f;
    auto join = [&](float2 o) {
        const float big = fmaxf(m, o.x);
        const float keep = m == big ? 1.0f : __expf(m - big), add = o.x == big ? 1.0f : __expf(o.x - big);
        s = s * keep + o.y * add;
        m = big;
    };
    if (row < p.rows) {
        for (int i = slice; i < p.parts; i += 128) {
            float2 o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                o[u] = i + 32 * u < p.parts ? p.stats[(size_t)(i + 32 * u) * p.rows + row] : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int u = 0; u < 4; ++u) join(o[u]);
        }
    }
    part[slice][l] = make_float2(m, s);
    __syncthreads();
    // warp w joins row w's 32 slices: in pairs, always the same ones
    const float2 mine = part[l][slice];
    m = mine.x;
    s = mine.y;
    __syncthreads();  // `part` is free again
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
        join(make_float2(om, os));
    }
    const int mine_row = blockIdx.x * 32 + slice;
    if (l == 0 && mine_row < p.rows) {
        const float lse = m + logf(s);
        const long long t = p.target[mine_row];
        p.lse[mine_row] = lse;
        const float loss = t == p.ignore_index ? 0.0f
                           : t < 0 || t >= p.vocab ? __int_as_float(0x7FC00000) : lse - p.target_logit[mine_row];
        p.row_loss[mine_row] = loss;
        if (p.total != nullptr) part[0][slice] = make_float2(loss, t != p.ignore_index ? 1.0f : 0.0f);
    }
    if (p.total == nullptr) return;
    __syncthreads();
    if (slice == 0) {
        float2 v = l < p.rows ? part[0][l] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if (l == 0) *p.total = p.mean ? (v.y > 0.0f ? v.x / v.y : 0.0f) : v.x;
    }
}

// All threads of a block of 32 warps: `join` over every thread's v, in a fixed order.
template <typename T, typename F>
__device__ __forceinline__ T block_join(T v, T* scratch, F join) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// loss = sum of the rows' losses, over the rows that count when mean.  One
// block; each thread sums every 1024th row with Kahan's compensation, then
// pairwise (fp64, which this GPU runs at a small fraction of fp32's rate, took 14.5
// us here; this takes 3).  A sum that is infinite has nothing to compensate: its
// difference to the terms would be NaN and spread to the rows that follow.
__global__ void __launch_bounds__(1024) layer_loss_sum_kernel(const float* row_loss, const long long* target, float* loss,
                                                             int rows, long long ignore_index, int mean) {
    __shared__ float fscratch[32];
    __shared__ int iscratch[32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float s = 0.0f, lost = 0.0f;
    int n = 0;
    for (int r = threadIdx.x; r < rows; r += 1024) {
        const float y = __fsub_rn(row_loss[r], lost), t = __fadd_rn(s, y);
        lost = isinf(t) ? 0.0f : __fsub_rn(__fsub_rn(t, s), y);
        s = t;
        n += target[r] != ignore_index;
    }
    s = block_join(s, fscratch, [](float a, float b) { return a + b; });
    n = block_join(n, iscratch, [](int a, int b) { return a + b; });
    if (threadIdx.x == 0) *loss = mean ? (n > 0 ? s / (float)n : 0.0f) : s;
}

// Each row's weight d loss / d row loss: grad[0] / rows that count (mean),
// grad[0] (sum) or grad[row] (none), relative to the largest and times 2^14: p
// times the largest weight then keeps fp16's full precision down to p = 2^-28 (unscaled, 1 /
// tokens times p is subnormal at once), and where all weights are alike a target's
// entry p - 1 rounds as itself, near -1 to next to nothing (with a power of two alone
// every target's entry took the same rounding of the weight, up to 0.4 % in bf16).
// Ignored rows weigh 0; a target that is no word makes its row's weight NaN.
// unscale = the largest weight over 2^14, for the products' epilogues.  That is right for dw,
// whose entries are sums over the rows.  A row of dh is its own weight's alone, and where the
// weights differ (none) fp16 loses the small p of a row far below the largest and all of one
// 2^-39 of it: there dh gets a d whose every row is scaled by 2^14 (row_weight: that, or 0 or
// NaN as above) and unscaled by row_unscale = the row's weight over 2^14.  (bf16 has the
// exponents.)  One block.
__global__ void __launch_bounds__(1024) layer_loss_weights_kernel(const float* grad, const long long* target, float* weight,
                                                                  float* unscale, float* row_weight, float* row_unscale,
                                                                  int rows, long long vocab, long long ignore_index,
                                                                  int reduction) {
    __shared__ float fscratch[32];
    __shared__ int iscratch[32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float most = 0.0f;
    int n = 0;
    for (int r = threadIdx.x; r < rows; r += 1024) {
        const bool counts = target[r] != ignore_index;
        n += counts;
        if (counts && reduction == 0) most = fmaxf(most, fabsf(grad[r]));
    }
    n = block_join(n, iscratch, [](int a, int b) { return a + b; });
    const float each = reduction == 0 ? 0.0f : reduction == 1 ? grad[0] / (float)max(n, 1) : grad[0];
    most = reduction == 0 ? block_join(most, fscratch, [](float a, float b) { return fmaxf(a, b); }) : fabsf(each);
    const bool scalable = most > 0.0f && most < INFINITY;  // else (0, inf, NaN) as it is
    for (int r = threadIdx.x; r < rows; r += 1024) {
        const long long t = target[r];
        const float w = reduction == 0 ? grad[r] : each;
        weight[r] = t == ignore_index ? 0.0f
                    : t < 0 || t >= vocab ? __int_as_float(0x7FC00000) : scalable ? __fdiv_rn(w, most) * 16384.0f : w;
        if (row_weight != nullptr) {
            row_weight[r] = t == ignore_index || w == 0.0f ? 0.0f : t < 0 || t >= vocab ? __int_as_float(0x7FC00000) : 16384.0f;
            row_unscale[r] = t == ignore_index ? 0.0f : w * (1.0f / 16384.0f);
        }
    }
    if (threadIdx.x == 0) *unscale = scalable ? most * (1.0f / 16384.0f) : 1.0f;
}

}  // namespace tcgemm
