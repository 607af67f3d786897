// Matrices into microscaled blocks, along their rows or their columns, and back.
// Bound by HBM: an element costs 2 bytes read and 1 1/32 or 1/2 + 1/32 written (back: 4096 x
// 14336 from 4 bits 24.2 us, 6.1 TB/s; 8192 x 4096 12.3 us, 6.9 TB/s).
#pragma once

#include "mx_common.cuh"

namespace tcgemm {

struct MxQuantParams {
    const void* x;
    uint8_t* data;
    uint32_t* scale;
    long long ldx, ldd;
    int rows, cols;       // of x
    int groups;           // blocks of threads along the columns
};

// Along the rows: a lane has eight neighbouring columns, a warp 256 of them, kMxQuantRows
// rows one after another with all their loads under way.  4096 x 14336 to 4 bits 25.9 us,
// 5.7 TB/s; 80 instructions for eight values take 60 % of what the SMs issue.  (With every
// row's addresses worked out by itself 108 of them, 30.4 us; eight rows a warp 31.2.)
constexpr int kMxQuantRows = 4;
static_assert(32 % kMxQuantRows == 0, "a warp's rows share a group of 32, their scale words 16 bytes apart");

template <int DT, int FMT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = blockIdx.x % p.groups, block = blockIdx.x / p.groups;
    const int col = group * 256 + lane * 8;
    const int k_tiles = (p.cols + 127) >> 7;
    const long long row0 = ((long long)block * 8 + warp) * kMxQuantRows;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (row0 >= p.rows) return;  // whole warps
    const int rows = (int)min((long long)kMxQuantRows, p.rows - row0);
    const unsigned short* src = static_cast<const unsigned short*>(p.x) + row0 * p.ldx + col;
    uint8_t* data = p.data + row0 * p.ldd + (FMT == kE4M3 ? col : col >> 1);
    uint32_t* word = p.scale + (mx_scale_word(row0, col >> 7, k_tiles) >> 2);
    const bool in_block = col < ((p.cols + 31) & ~31), in_word = (col >> 7) < k_tiles;
    uint4 v[kMxQuantRows];
    if (rows == kMxQuantRows && (group + 1) * 256ll <= p.cols) {
#pragma unroll
        for (int u = 0; u < kMxQuantRows; ++u) v[u] = *reinterpret_cast<const uint4*>(src + u * p.ldx);
    } else {
#pragma unroll
        for (int u = 0; u < kMxQuantRows; ++u)
            v[u] = u < rows && col < p.cols ? load8<DT>(src, u * p.ldx, col, p.cols) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kMxQuantRows; ++u) {
        if (u >= rows) break;
        float f[8];
        unpack8<DT>(v[u], f);
        const uint32_t m2 = max_abs2(max_abs2(max_abs2(v[u].x & 0x7FFF7FFFu, v[u].y), v[u].z), v[u].w);
        mx_store8<FMT>(f, max_half_bits<DT>(m2), data + u * p.ldd, in_block, word + 4 * u, in_word);
    }
}

// Along the columns, result [cols, rows]: a CTA has 128 rows x 128 columns, a thread two
// neighbouring columns of 32 rows, so that a block never leaves its registers and a warp
// reads 128 bytes of each row.  A column's four blocks meet in shared memory, from where
// they go out side by side, 64 or 128 bytes.  4096 x 14336 to 4 bits 23.6 us, 6.3 TB/s (a
// thread on four blocks one after another, stored as they came: 33.6).
template <int DT, int FMT>
__global__ void __launch_bounds__(256) mx_quantize_columns_kernel(const MxQuantParams p) {
    constexpr int kBytes = mx_block_bytes(FMT), kPieces = 4 * kBytes / 16;  // 16-byte pieces of a column
    __shared__ uint4 out[128][kPieces + 1];
    __shared__ __align__(4) uint8_t bytes[128][4];
    const long long group = blockIdx.x % p.groups, tile = blockIdx.x / p.groups;
    const int lane = threadIdx.x & 31, b = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7;
    const int c0 = half * 64 + lane * 2;
    const long long col = group * 128 + c0, r0 = tile * 128 + b * 32;
    const int k_tiles = (p.rows + 127) >> 7;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const bool one = col < p.cols, two = col + 1 < p.cols;
    const unsigned short* src = static_cast<const unsigned short*>(p.x) + r0 * p.ldx + col;
    uint32_t v[32];
    if (r0 + 32 <= p.rows && (group + 1) * 128 <= p.cols) {
#pragma unroll
        for (int i = 0; i < 32; ++i, src += p.ldx) v[i] = *reinterpret_cast<const uint32_t*>(src);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v[i] = 0u;
            if (r0 + i < p.rows) {
                if (two)
                    v[i] = *reinterpret_cast<const uint32_t*>(src + i * p.ldx);
                else if (one)
                    v[i] = src[i * p.ldx];
            }
        }
    }
    uint32_t m2 = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) m2 = max_abs2(m2, v[i]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t byte = mx_scale_byte<FMT>(max_half_bits<DT>(c == 0 ? m2 & 0xFFFFu : m2 >> 16));
        const float un = mx_unscale(byte);
        bytes[c0 + c][b] = (uint8_t)byte;
        uint2 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 pair = unpack2<DT>(v[8 * j + i]);
                f[i] = c == 0 ? pair.x : pair.y;
            }
            q[j] = mx_pack8<FMT>(f, un);
        }
        if constexpr (FMT == kE4M3) {
            out[c0 + c][2 * b] = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
            out[c0 + c][2 * b + 1] = make_uint4(q[2].x, q[2].y, q[3].x, q[3].y);
        } else {
            out[c0 + c][b] = make_uint4(q[0].x, q[1].x, q[2].x, q[3].x);
        }
    }
    __syncthreads();
    // pieces of rows that exist: up to the end of the last block
    const int pieces = (int)min((long long)kPieces, ((p.rows + 31ll) / 32 - tile * 4) * (kBytes / 16));
#pragma unroll
    for (int i = threadIdx.x; i < 128 * kPieces; i += 256) {
        const int c = i / kPieces, piece = i % kPieces;
        if (group * 128 + c < p.cols && piece < pieces)
            *reinterpret_cast<uint4*>(p.data + (group * 128 + c) * p.ldd + tile * (4 * kBytes) + piece * 16) = out[c][piece];
    }
    if (threadIdx.x < 128 && group * 128 + threadIdx.x < p.cols)
        p.scale[mx_scale_word(group * 128 + threadIdx.x, tile, k_tiles) >> 2] = *reinterpret_cast<const uint32_t*>(bytes[threadIdx.x]);
}

struct MxValuesParams {
    const uint8_t* data;
    const uint8_t* scale;
    void* x;
    long long ldd, ldx;
    int rows, cols;
    int groups;
};

// Back into 16 bits, laid out as mx_quantize_kernel.
template <int DT, int FMT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxValuesParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long group = blockIdx.x % p.groups, block = blockIdx.x / p.groups;
    const int col = (int)(group * 256) + lane * 8;
    const int k_tiles = (p.cols + 127) >> 7;
    const long long row0 = (block * 8 + warp) * kMxQuantRows;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (col >= p.cols) return;
    uint2 q[kMxQuantRows];
    uint32_t s[kMxQuantRows];
#pragma unroll
    for (int u = 0; u < kMxQuantRows; ++u) {
        const long long row = row0 + u;
        if (row >= p.rows) break;
        const uint8_t* d = p.data + row * p.ldd + (FMT == kE4M3 ? col : col >> 1);
        if constexpr (FMT == kE4M3)
            q[u] = *reinterpret_cast<const uint2*>(d);
        else
            q[u] = make_uint2(*reinterpret_cast<const uint32_t*>(d), 0u);
        s[u] = p.scale[mx_scale_word(row, col >> 7, k_tiles) + ((col >> 5) & 3)];
    }
#pragma unroll
    for (int u = 0; u < kMxQuantRows; ++u) {
        const long long row = row0 + u;
        if (row >= p.rows) break;
        float f[8];
        mx_unpack8<FMT>(q[u], mx_scale_value(s[u]), f);
        store8(p.x, row * p.ldx + col, col, p.cols, pack8<DT>(f));
    }
}

}  // namespace tcgemm
