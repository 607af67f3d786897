// The root-mean-square norm with the residual's addition, its output in 16 bits or
// in microscaled blocks, and its gradients.
//
//   h = x + residual,  r = 1 / sqrt(mean h^2 + eps),  y = h r w
//   dx = r (dy w) - h r^3 mean(dy w h) + dh,  dw = sum over rows of dy h r
//
// Bound by HBM: every matrix is read or written once.  A row's values stay in the
// registers of the threads that share it, eight neighbouring columns (16 bytes) to
// a load, between the sum over the row and its use; rows beyond 32768 columns
// forward and 16384 back are read twice instead.  All sums are fp32 and taken in a
// fixed order: the same inputs give the same bits.  8192 x 4096 in bf16 with residual
// 40.8 us, 6.6 TB/s of 268 MB; gradients 47.6, 5.6 TB/s, of which the join of dweight's
// partial sums takes some 4.
#pragma once

#include "mx_common.cuh"

namespace tcgemm {

enum NormOut { kNormRow = 0, kNormE4M3 = 1, kNormE2M1 = 2 };

struct NormParams {
    const void *x, *residual, *weight;
    void *h, *y;
    uint8_t* data;
    uint32_t* scale;
    float* rstd;
    long long ldx, ldr, ldh, ldy, ldd;
    int tokens, dim;
    int group;       // threads that share a row: 32 or all of a block's
    float eps;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

__device__ __forceinline__ float norm_rstd(float squares, int dim, float eps) {
    return __frsqrt_rn(__fdiv_rn(squares, (float)dim) + eps);
}

// Where a row of the outputs begins.
struct NormRowOut {
    unsigned short* y;
    uint8_t* data;
    uint32_t* scale;  // the first tile's word of this row; the next tile's is 128 words on
};

template <int OUT>
__device__ __forceinline__ NormRowOut norm_row_out(const NormParams& p, int row) {
    NormRowOut o{p.y != nullptr ? static_cast<unsigned short*>(p.y) + row * p.ldy : nullptr, nullptr, nullptr};
    if constexpr (OUT != kNormRow) {
        o.data = p.data + row * p.ldd;
        o.scale = p.scale + (mx_scale_word(row, 0, (p.dim + 127) >> 7) >> 2);
    }
    return o;
}

// Eight columns of y: scaled, and stored in each form that is wanted.
template <int DT, int OUT>
__device__ __forceinline__ void norm_store(const NormParams& p, const NormRowOut& o, int col, uint4 hv, float rstd) {
    float h[8], w[8], f[8];
    unpack8<DT>(hv, h);
    unpack8<DT>(col < p.dim ? load8<DT>(p.weight, col, col, p.dim) : make_uint4(0u, 0u, 0u, 0u), w);
    // h w is exact in fp32 (two 16-bit significands), so y is rounded once before its last rounding
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 two = parts(mul2(mul2(f2(h[i], h[i + 1]), f2(w[i], w[i + 1])), both(rstd)));
        f[i] = two.x;
        f[i + 1] = two.y;
    }
    if (o.y != nullptr && col < p.dim) store8(o.y, col, col, p.dim, pack8<DT>(f));
    if constexpr (OUT != kNormRow) {
        constexpr int kFmt = OUT == kNormE4M3 ? kE4M3 : kE2M1;
        if (col + 8 > p.dim) {  // behind the row's end h and w are 0, but rstd may be infinite
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i >= p.dim) f[i] = 0.0f;
        }
        uint32_t m = abs_bits(f[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, abs_bits(f[i]));
        mx_store8<kFmt>(f, m, o.data + (kFmt == kE4M3 ? col : col >> 1), col < ((p.dim + 31) & ~31), o.scale + (col >> 7) * 128,
                        (col >> 7) < ((p.dim + 127) >> 7));
    }
}

// V vectors of eight columns a thread: thread t of a row's group has columns 8 (t + j group).
template <int DT, int V, int OUT>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
    __shared__ float sums[32];
    const int lane = threadIdx.x & 31;
    const bool alone = p.group == 32;  // a warp a row
    const int t = alone ? lane : (int)threadIdx.x;
    const int row = alone ? (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) : (int)blockIdx.x;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (row >= p.tokens) return;  // whole warps
    uint4 h[V], r[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int col = (t + j * p.group) * 8;
        h[j] = col < p.dim ? load8<DT>(p.x, row * p.ldx + col, col, p.dim) : make_uint4(0u, 0u, 0u, 0u);
        if (p.residual != nullptr)
            r[j] = col < p.dim ? load8<DT>(p.residual, row * p.ldr + col, col, p.dim) : make_uint4(0u, 0u, 0u, 0u);
    }
    float squares = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int col = (t + j * p.group) * 8;
        float a[8];
        unpack8<DT>(h[j], a);
        if (p.residual != nullptr) {
            float b[8];
            unpack8<DT>(r[j], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += b[i];
            h[j] = pack8<DT>(a);
            unpack8<DT>(h[j], a);  // as it is stored
            if (col < p.dim) store8(p.h, row * p.ldh + col, col, p.dim, h[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = fmaf(a[i], a[i], squares);
    }
    squares = warp_sum(squares);
    if (!alone) {
        if (lane == 0) sums[threadIdx.x >> 5] = squares;
        __syncthreads();
        squares = warp_sum(lane < (int)(blockDim.x >> 5) ? sums[lane] : 0.0f);
    }
    const float rstd = norm_rstd(squares, p.dim, p.eps);
    if (t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    __syncwarp();
    const NormRowOut o = norm_row_out<OUT>(p, row);
#pragma unroll
    for (int j = 0; j < V; ++j) norm_store<DT, OUT>(p, o, (t + j * p.group) * 8, h[j], rstd);
}

// Rows too long for registers, a block of 1024 threads each: h is written in the first
// pass and read again in the second (by the thread that wrote it).
template <int DT, int OUT>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const NormParams p) {
    __shared__ float sums[32];
    const int lane = threadIdx.x & 31;
    const int row = (int)blockIdx.x;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float squares = 0.0f;
    for (long long c = threadIdx.x * 8; c < p.dim; c += 8192) {
        const int col = (int)c;
        float a[8];
        unpack8<DT>(load8<DT>(p.x, row * p.ldx + col, col, p.dim), a);
        if (p.residual != nullptr) {
            float b[8];
            unpack8<DT>(load8<DT>(p.residual, row * p.ldr + col, col, p.dim), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += b[i];
            const uint4 h = pack8<DT>(a);
            unpack8<DT>(h, a);
            store8(p.h, row * p.ldh + col, col, p.dim, h);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = fmaf(a[i], a[i], squares);
    }
    squares = warp_sum(squares);
    if (lane == 0) sums[threadIdx.x >> 5] = squares;
    __syncthreads();
    squares = warp_sum(sums[lane]);
    const float rstd = norm_rstd(squares, p.dim, p.eps);
    if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    __syncwarp();
    const void* src = p.residual != nullptr ? p.h : p.x;
    const long long ld = p.residual != nullptr ? p.ldh : p.ldx;
    const NormRowOut o = norm_row_out<OUT>(p, row);
    // whole warps to the end of the last block's tile
    for (long long c = (long long)(threadIdx.x - lane) * 8; c < (p.dim + 127ll & ~127ll); c += 8192) {
        const int col = (int)c + lane * 8;
        const uint4 h = col < p.dim ? load8<DT>(src, row * ld + col, col, p.dim) : make_uint4(0u, 0u, 0u, 0u);
        norm_store<DT, OUT>(p, o, col, h, rstd);
    }
}

// ---- gradients ---------------------------------------------------------------------------

// Blocks of the gradients are counted for this many SMs whatever the device has: the workspace
// for their sums of dweight is sized on the host, without a device, and the order of those sums,
// with it the result's bits, is the same everywhere.
constexpr int kNormSms = 152;

struct NormGradParams {
    const void *dy, *h, *weight, *dh;
    const float* rstd;
    void* dx;
    float* partial;    // rows of pitch() sums, one a block; NULL where dweight is not wanted
    long long lddy, ldh, lddh, lddx;
    int tokens, dim;
    __host__ __device__ size_t pitch() const { return ((size_t)dim + 7) & ~(size_t)7; }
};

__device__ __forceinline__ void store_sums(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// 16 bytes into shared memory, of which `bytes` are read and the rest is 0.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
    uint4 v;
    ptx::ld_shared_v4(at, v.x, v.y, v.z, v.w);
    return v;
}

// A block's threads share the columns, two vectors of eight each, and walk over the rows,
// their share of dweight in registers.  What a thread will need of the next DEPTH - 1 rows is
// on its way into shared memory, where only that thread reads it: nobody waits for loads at
// the barrier in a row's sum, and 512 threads an SM have 150 KB under way.  (With the loads in
// registers, 8192 x 4096: one to four blocks an SM 53 to 88 us.)
template <int DT, int DEPTH, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rms_norm_grad_kernel(const NormGradParams p) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float sums[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t mine = ptx::smem_addr(ring) + threadIdx.x * 16u, vector = blockDim.x * 16u;
    auto slot = [&](int stage, int which, int j) { return mine + (uint32_t)((stage * 3 + which) * 2 + j) * vector; };
    const int cols[2] = {(int)threadIdx.x * 8, (int)(threadIdx.x + blockDim.x) * 8};
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float dw[2][8];
    uint4 w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        w[j] = cols[j] < p.dim ? load8<DT>(p.weight, cols[j], cols[j], p.dim) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    }
    auto fetch = [&](long long row, int stage) {
        if (row < p.tokens) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int bytes = min(16, (p.dim - cols[j]) * 2);
                if (bytes > 0) {
                    copy_async16(slot(stage, 0, j), static_cast<const unsigned short*>(p.dy) + row * p.lddy + cols[j], bytes);
                    copy_async16(slot(stage, 1, j), static_cast<const unsigned short*>(p.h) + row * p.ldh + cols[j], bytes);
                    if (p.dh != nullptr)
                        copy_async16(slot(stage, 2, j), static_cast<const unsigned short*>(p.dh) + row * p.lddh + cols[j], bytes);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const long long step = gridDim.x;
    for (int i = 0; i < DEPTH - 1; ++i) fetch(blockIdx.x + i * step, i);
    int stage = 0, set = 0;
    float next_rstd = blockIdx.x < (unsigned)p.tokens ? p.rstd[blockIdx.x] : 0.0f;
    for (long long row = blockIdx.x; row < p.tokens; row += step, set ^= 1) {
        fetch(row + (DEPTH - 1) * step, stage == 0 ? DEPTH - 1 : stage - 1);
        const float rstd = next_rstd;
        if (row + step < p.tokens) next_rstd = p.rstd[row + step];
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (cols[j] >= p.dim) continue;
            float a[8], b[8], c[8];
            unpack8<DT>(ld_shared16(slot(stage, 0, j)), a);
            unpack8<DT>(ld_shared16(slot(stage, 1, j)), b);
            unpack8<DT>(w[j], c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dot = fmaf(a[i] * c[i], b[i], dot);
                dw[j][i] = fmaf(a[i] * b[i], rstd, dw[j][i]);
            }
        }
        if (p.dx != nullptr) {
            dot = warp_sum(dot);
            if (lane == 0) sums[set][warp] = dot;
            __syncthreads();
            const float back = __fdiv_rn(warp_sum(lane < warps ? sums[set][lane] : 0.0f), (float)p.dim) * rstd * rstd * rstd;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (cols[j] >= p.dim) continue;
                float a[8], b[8], c[8], d[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                unpack8<DT>(ld_shared16(slot(stage, 0, j)), a);
                unpack8<DT>(ld_shared16(slot(stage, 1, j)), b);
                unpack8<DT>(w[j], c);
                if (p.dh != nullptr) unpack8<DT>(ld_shared16(slot(stage, 2, j)), d);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] += fmaf(a[i] * c[i], rstd, -b[i] * back);
                store8(p.dx, row * p.lddx + cols[j], cols[j], p.dim, pack8<DT>(d));
            }
        }
        if (++stage == DEPTH) stage = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (p.partial == nullptr) return;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (cols[j] < p.dim) store_sums(p.partial + blockIdx.x * p.pitch() + cols[j], dw[j]);
}

// dx of rows too long for the above, a block of 1024 threads each, in two passes.
template <int DT>
__global__ void __launch_bounds__(1024) rms_norm_grad_long_kernel(const NormGradParams p) {
    __shared__ float sums[32];
    const int lane = threadIdx.x & 31;
    const long long row = blockIdx.x;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const float rstd = p.rstd[row];
    float dot = 0.0f;
    for (long long c = threadIdx.x * 8; c < p.dim; c += 8192) {
        const int col = (int)c;
        float a[8], b[8], w[8];
        unpack8<DT>(load8<DT>(p.dy, row * p.lddy + col, col, p.dim), a);
        unpack8<DT>(load8<DT>(p.h, row * p.ldh + col, col, p.dim), b);
        unpack8<DT>(load8<DT>(p.weight, col, col, p.dim), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(a[i] * w[i], b[i], dot);
    }
    dot = warp_sum(dot);
    if (lane == 0) sums[threadIdx.x >> 5] = dot;
    __syncthreads();
    const float back = __fdiv_rn(warp_sum(sums[lane]), (float)p.dim) * rstd * rstd * rstd;
    for (long long c = threadIdx.x * 8; c < p.dim; c += 8192) {
        const int col = (int)c;
        float a[8], b[8], w[8], d[8];
        unpack8<DT>(load8<DT>(p.dy, row * p.lddy + col, col, p.dim), a);
        unpack8<DT>(load8<DT>(p.h, row * p.ldh + col, col, p.dim), b);
        unpack8<DT>(load8<DT>(p.weight, col, col, p.dim), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(a[i] * w[i], rstd, -b[i] * back);
        if (p.dh != nullptr) {
            float e[8];
            unpack8<DT>(load8<DT>(p.dh, row * p.lddh + col, col, p.dim), e);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] += e[i];
        }
        store8(p.dx, row * p.lddx + col, col, p.dim, pack8<DT>(d));
    }
}

// dweight's partial sums for such rows: a thread on eight columns (blockIdx.x), a share of
// the rows a block (blockIdx.y).
template <int DT>
__global__ void __launch_bounds__(256) rms_norm_grad_columns_kernel(const NormGradParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int col = (int)(blockIdx.x * 256 + threadIdx.x) * 8;
    if (col >= p.dim) return;
    const long long r0 = (long long)p.tokens * blockIdx.y / gridDim.y, r1 = (long long)p.tokens * (blockIdx.y + 1) / gridDim.y;
    float dw[8] = {};
#pragma unroll 4
    for (long long row = r0; row < r1; ++row) {
        const float rstd = p.rstd[row];
        float a[8], b[8];
        unpack8<DT>(load8<DT>(p.dy, row * p.lddy + col, col, p.dim), a);
        unpack8<DT>(load8<DT>(p.h, row * p.ldh + col, col, p.dim), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] = fmaf(a[i] * b[i], rstd, dw[i]);
    }
    store_sums(p.partial + blockIdx.y * p.pitch() + col, dw);
}

// dweight[c] = sum over blocks of their sums of column c, rounded once: 32 columns a block
// (a warp reads 128 bytes), 32 slices of the partials side by side, eight reads under way.
template <int DT>
__global__ void __launch_bounds__(1024) rms_norm_weight_sum_kernel(const NormGradParams p, void* out, int blocks) {
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const long long c = blockIdx.x * 32ll + lane;
    const size_t pitch = p.pitch();
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float s = 0.0f;
    if (c < p.dim) {
        for (int b = slice; b < blocks; b += 256) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = b + 32 * i < blocks ? __ldcg(p.partial + (b + 32 * i) * pitch + c) : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
    }
    sums[slice][lane] = s;
    __syncthreads();
    s = warp_sum(sums[lane][slice]);
    const long long mine = blockIdx.x * 32ll + slice;
    if (lane == 0 && mine < p.dim) static_cast<unsigned short*>(out)[mine] = pack1<DT>(s);
}

}  // namespace tcgemm
