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
__global__ void __launch_bounds__(256) layer_slope_kernel(const SlopeParams p) {
    __shared__ float sums[8][kSlopeCols];
    const int cg = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int cb = blockIdx.x % p.col_blocks, rb = blockIdx.x / p.col_blocks;
    const int col = cb * kSlopeCols + cg * 8;
    const int r0 = rb * kSlopeRows;
    const int r1 = min(p.rows, r0 + kSlopeRows);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (col < p.cols) {
        const bool whole = col + 8 <= p.cols;
        with_act(p.pre ? p.act : kActNone, [&](auto tag) {
            constexpr int ACT = decltype(tag)::value;
#pragma unroll 2
            for (int r = r0 + rl; r < r1; r += 8) {
                const unsigned short* dy = static_cast<const unsigned short*>(p.dy) + r * p.ld_dy + col;
                const unsigned short* pre = static_cast<const unsigned short*>(p.pre) + r * p.ld_pre + col;
                float d[8];
                if (whole) {
                    const uint4 w = *reinterpret_cast<const uint4*>(dy);
                    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = unpack2<DT>(ws[e]);
                        d[2 * e] = f.x;
                        d[2 * e + 1] = f.y;
                    }
                    if constexpr (ACT != kActNone) {
                        const uint4 z = *reinterpret_cast<const uint4*>(pre);
                        const uint32_t zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = unpack2<DT>(zs[e]);
                            d[2 * e] *= act_slope<ACT>(f.x);
                            d[2 * e + 1] *= act_slope<ACT>(f.y);
                        }
                    }
                    if (p.dpre)
                        *reinterpret_cast<uint4*>(static_cast<unsigned short*>(p.dpre) + r * p.ld_dpre + col) =
                            make_uint4(pack2<DT>(d[0], d[1]), pack2<DT>(d[2], d[3]), pack2<DT>(d[4], d[5]),
                                       pack2<DT>(d[6], d[7]));
                } else {
                    for (int e = 0; e < 8; ++e) {
                        d[e] = 0.0f;
                        if (col + e >= p.cols) continue;
                        d[e] = load1<DT>(dy, e);
                        if constexpr (ACT != kActNone) d[e] *= act_slope<ACT>(load1<DT>(pre, e));
                        if (p.dpre) static_cast<unsigned short*>(p.dpre)[r * p.ld_dpre + col + e] = pack1<DT>(d[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += d[e];
            }
        });
    }
    if (p.partial == nullptr) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[rl][cg * 8 + e] = acc[e];
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
};

// lse = max + ln(sum over parts of s_i exp(m_i - max)); loss = lse - target's
// logit.  An ignored row's loss is 0; a target that is neither ignored nor a
// word makes its row's loss NaN.  32 rows a block, 8 slices of the parts.
__global__ void __launch_bounds__(256) layer_loss_rows_kernel(const LossParams p) {
    __shared__ float2 part[8][32];
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
    if (row < p.rows)
        for (int i = slice; i < p.parts; i += 8) join(p.stats[(size_t)i * p.rows + row]);
    part[slice][l] = make_float2(m, s);
    __syncthreads();
    if (slice != 0 || row >= p.rows) return;
    m = -INFINITY;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) join(part[i][l]);
    const float lse = m + logf(s);
    const long long t = p.target[row];
    p.lse[row] = lse;
    p.row_loss[row] = t == p.ignore_index ? 0.0f
                      : t < 0 || t >= p.vocab ? __int_as_float(0x7FC00000) : lse - p.target_logit[row];
}

template <typename T, typename F>
__device__ __forceinline__ T block_join(T v, T* scratch, F join) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
    for (int i = 1; i < (int)(blockDim.x >> 5); ++i) v = join(v, scratch[i]);
    return v;
}

// loss = sum of the rows' losses, over the rows that count when mean.  One
// block; each thread sums its rows in order, in fp64 (rows / 1024 additions).
__global__ void __launch_bounds__(1024) layer_loss_sum_kernel(const float* row_loss, const long long* target, float* loss,
                                                             int rows, long long ignore_index, int mean) {
    __shared__ double dsum[32];
    __shared__ int isum[32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    double s = 0.0;
    int n = 0;
    for (int r = threadIdx.x; r < rows; r += 1024) {
        s += (double)row_loss[r];
        n += target[r] != ignore_index;
    }
    s = block_join(s, dsum, [](double a, double b) { return a + b; });
    n = block_join(n, isum, [](int a, int b) { return a + b; });
    if (threadIdx.x == 0) *loss = (float)(mean ? (n > 0 ? s / n : 0.0) : s);
}

// Each row's weight d loss / d row loss: grad[0] / rows that count (mean),
// grad[0] (sum) or grad[row] (none), times a power of two that puts the largest
// in [2^14, 2^15): p times the weight then keeps fp16's full precision down to
// p = 2^-28 (unscaled, 1 / tokens times p is subnormal at once).  Ignored
// rows weigh 0; a target that is no word makes its row's weight NaN.  unscale =
// the power's inverse, for the products' epilogues.  One block.
__global__ void __launch_bounds__(1024) layer_loss_weights_kernel(const float* grad, const long long* target, float* weight,
                                                                  float* unscale, int rows, long long vocab,
                                                                  long long ignore_index, int reduction) {
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
    // 2^e <= most < 2^(e+1); 0, inf and NaN are left unscaled
    const int e = (int)((__float_as_uint(most) >> 23) & 255) - 127;
    const bool scalable = most > 0.0f && e > -127 && e < 128;
    const int up = scalable ? min(max(14 - e, -100), 100) : 0;
    const float scale = __uint_as_float((uint32_t)(127 + up) << 23);
    for (int r = threadIdx.x; r < rows; r += 1024) {
        const long long t = target[r];
        const float w = (reduction == 0 ? grad[r] : each) * scale;
        weight[r] = t == ignore_index ? 0.0f : t < 0 || t >= vocab ? __int_as_float(0x7FC00000) : w;
    }
    if (threadIdx.x == 0) *unscale = __uint_as_float((uint32_t)(127 - up) << 23);
}

}  // namespace tcgemm
