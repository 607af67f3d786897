// Microscaled matrices (include/mx_ops.h): the two element formats, the blocks'
// scales and where they lie, and the conversion of eight values of a block that
// four neighbouring lanes hold.
#pragma once

#include "layer_common.cuh"

namespace tcgemm {

enum MxFormat { kE4M3 = 0, kE2M1 = 1 };

constexpr int kMxBlock = 32;                      // values that share a scale
__host__ __device__ constexpr int mx_emax(int fmt) { return fmt == kE4M3 ? 8 : 2; }
__host__ __device__ constexpr int mx_block_bytes(int fmt) { return fmt == kE4M3 ? 32 : 16; }

// The word that holds the scales of four blocks (4 k4 ..) of one row, k_tiles tiles a
// row of tiles.
__host__ __device__ __forceinline__ long long mx_scale_word(long long row, long long k4, long long k_tiles) {
    return ((row >> 7) * k_tiles + k4) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Scale byte of a block whose largest magnitude has these bits (an fp32's, without its
// sign; an infinity's or a NaN's are the largest): floor(log2 amax) is the exponent field
// itself, so the byte is that less emax, 0 at least.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    const uint32_t e = amax >> 23;
    return e == 255u ? 255u : e > (uint32_t)mx_emax(FMT) ? e - mx_emax(FMT) : 0u;
}

// 1 / scale, exact: 2^(127 - byte).  (Byte 255 gives 0, with which nothing is NaN or not
// that the scale does not make NaN anyway.)
__device__ __forceinline__ float mx_unscale(uint32_t byte) {
    return byte >= 254u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// Eight values to the format, nearest even, saturated: one word (e2m1) or two (e4m3).
template <int FMT>
__device__ __forceinline__ uint2 mx_pack8(const float (&f)[8], float unscale) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 two = parts(mul2(f2(f[i], f[i + 1]), both(unscale)));
        v[i] = two.x;
        v[i + 1] = two.y;
    }
    if constexpr (FMT == kE4M3) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            unsigned short lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * i + 1]), "f"(v[4 * i]));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * i + 3]), "f"(v[4 * i + 2]));
            w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
        return make_uint2(w[0], w[1]);
    } else {
        uint32_t w;
        asm("{\n"
            "  .reg .b8 a, b, c, d;\n"
            "  cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
            "  cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
            "  cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
            "  cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
            "  mov.b32 %0, {a, b, c, d};\n"
            "}\n"
            : "=r"(w)
            : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
        return make_uint2(w, 0u);
    }
}

// Eight values of a microscaled row, from the words mx_pack8 made; scale as a factor.
// e2m1 goes by way of fp16 pairs, which hold its values exactly, as they do e4m3's.
template <int FMT>
__device__ __forceinline__ void mx_unpack8(uint2 w, float scale, float (&f)[8]) {
    uint32_t h[4];
    if constexpr (FMT == kE4M3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned short two = (unsigned short)((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"(two));
        }
    } else {
        asm("{\n"
            "  .reg .b8 a, b, c, d;\n"
            "  mov.b32 {a, b, c, d}, %4;\n"
            "  cvt.rn.f16x2.e2m1x2 %0, a;\n"
            "  cvt.rn.f16x2.e2m1x2 %1, b;\n"
            "  cvt.rn.f16x2.e2m1x2 %2, c;\n"
            "  cvt.rn.f16x2.e2m1x2 %3, d;\n"
            "}\n"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w.x));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2<kF16>(h[i]);
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

// 2^(byte - 127) as a factor: byte 0 is fp32's subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
    return byte == 0u ? __uint_as_float(0x00400000u) : byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// The larger of two magnitudes in each half of two words of 16-bit values: their bits
// without the sign are ordered as whole numbers, NaN above infinity.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7FFF7FFFu); }

// The larger half of such a word as an fp32's bits.
template <int DT>
__device__ __forceinline__ uint32_t max_half_bits(uint32_t m) {
    const uint32_t one = max(m & 0xFFFFu, m >> 16);
    if constexpr (DT == kBF16) return one << 16;
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)one)));
}

// Four lanes hold a block of 32 values between them, eight each, m the bits of the largest
// magnitude of this lane's; sixteen lanes hold four blocks.  Stores the lane's eight at
// `data` (skipped where the block does not exist) and, from the first of the sixteen, their
// four scales at `word`.  Every lane of the warp calls this.
template <int FMT>
__device__ __forceinline__ void mx_store8(const float (&f)[8], uint32_t m, uint8_t* data, bool in_block, uint32_t* word, bool in_word) {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t byte = mx_scale_byte<FMT>(m);
    const uint2 w = mx_pack8<FMT>(f, mx_unscale(byte));
    if (in_block) {
        if constexpr (FMT == kE4M3)
            *reinterpret_cast<uint2*>(data) = w;
        else
            *reinterpret_cast<uint32_t*>(data) = w.x;
    }
    uint32_t all = byte << (8 * ((threadIdx.x >> 2) & 3));
    all |= __shfl_xor_sync(0xffffffffu, all, 4);
    all |= __shfl_xor_sync(0xffffffffu, all, 8);
    if (in_word && (threadIdx.x & 15) == 0) *word = all;
}

// Eight 16-bit values of a row from column `col` on, those from `cols` on absent (0).
template <int DT>
__device__ __forceinline__ uint4 load8(const void* p, long long at, int col, int cols) {
    if (col + 8 <= cols) return *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(p) + at);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < cols) w[e >> 1] |= (uint32_t)static_cast<const unsigned short*>(p)[at + e] << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(void* p, long long at, int col, int cols, uint4 v) {
    if (col + 8 <= cols) {
        *reinterpret_cast<uint4*>(static_cast<unsigned short*>(p) + at) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < cols) static_cast<unsigned short*>(p)[at + e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
}

template <int DT>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 two = unpack2<DT>(w[i]);
        f[2 * i] = two.x;
        f[2 * i + 1] = two.y;
    }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
}

}  // namespace tcgemm
