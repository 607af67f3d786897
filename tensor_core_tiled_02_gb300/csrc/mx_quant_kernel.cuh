// Matrices into microscaled blocks, along their rows or their columns, and back.
// Bound by HBM: an element costs 2 bytes read and 1 1/32 or 1/2 + 1/32 written.
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
// rows one after another with all their loads under way.
constexpr int kMxQuantRows = 4;
template <int DT, int FMT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long group = blockIdx.x % p.groups, block = blockIdx.x / p.groups;
    const int col = (int)(group * 256) + lane * 8;
    const int k_tiles = (p.cols + 127) >> 7;
    const long long row0 = (block * 8 + warp) * kMxQuantRows;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    uint4 v[kMxQuantRows];
#pragma unroll
    for (int u = 0; u < kMxQuantRows; ++u)
        v[u] = row0 + u < p.rows && col < p.cols ? load8<DT>(p.x, (row0 + u) * p.ldx + col, col, p.cols) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < kMxQuantRows; ++u) {
        const long long row = row0 + u;
        if (row >= p.rows) break;  // whole warps
        float f[8];
        unpack8<DT>(v[u], f);
        uint8_t* data = p.data + row * p.ldd + (FMT == kE4M3 ? col : col >> 1);
        uint32_t* word = p.scale + (mx_scale_word(row, col >> 7, k_tiles) >> 2);
        mx_store8<FMT>(f, data, col < ((p.cols + 31) & ~31), word, (col >> 7) < k_tiles);
    }
}

// Along the columns, result [cols, rows]: a thread has two neighbouring columns and 128
// rows of them, a block of 32 at a time, so that a block never leaves its registers and a
// warp reads 128 bytes of each row.
template <int DT, int FMT>
__global__ void __launch_bounds__(128) mx_quantize_columns_kernel(const MxQuantParams p) {
    const long long group = blockIdx.x % p.groups, tile = blockIdx.x / p.groups;
    const long long col = (group * 128 + threadIdx.x) * 2;
    const int k_tiles = (p.rows + 127) >> 7;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    if (col >= p.cols) return;
    const bool two = col + 1 < p.cols;
    const unsigned short* src = static_cast<const unsigned short*>(p.x) + col;
    uint32_t words[2] = {0u, 0u};
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
        const long long r0 = tile * 128 + b * 32;
        if (r0 >= p.rows) break;
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v[i] = 0u;
            if (r0 + i < p.rows)
                v[i] = two ? *reinterpret_cast<const uint32_t*>(src + (r0 + i) * p.ldx) : (uint32_t)src[(r0 + i) * p.ldx];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float f[4][8];
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float2 pair = unpack2<DT>(v[i]);
                f[i >> 3][i & 7] = c == 0 ? pair.x : pair.y;
                m = max(m, abs_bits(f[i >> 3][i & 7]));
            }
            if (c == 1 && !two) break;
            const uint32_t byte = mx_scale_byte<FMT>(m);
            const float un = mx_unscale(byte);
            words[c] |= byte << (8 * b);
            uint32_t* d = reinterpret_cast<uint32_t*>(p.data + (col + c) * p.ldd + (r0 >> 5) * mx_block_bytes(FMT));
            uint2 q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = mx_pack8<FMT>(f[i], un);
            if constexpr (FMT == kE4M3) {
                reinterpret_cast<uint4*>(d)[0] = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
                reinterpret_cast<uint4*>(d)[1] = make_uint4(q[2].x, q[2].y, q[3].x, q[3].y);
            } else {
                reinterpret_cast<uint4*>(d)[0] = make_uint4(q[0].x, q[1].x, q[2].x, q[3].x);
            }
        }
    }
    p.scale[mx_scale_word(col, tile, k_tiles) >> 2] = words[0];
    if (two) p.scale[mx_scale_word(col + 1, tile, k_tiles) >> 2] = words[1];
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
