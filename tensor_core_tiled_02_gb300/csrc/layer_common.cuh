// Pieces shared by the layer operators' kernels (linear layer, gated
// feed-forward block, vocabulary cross entropy): 16-bit element types,
// activations and their slopes, matrix descriptors for either major order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "gemm_common.cuh"

namespace tcgemm {

constexpr unsigned kSiteAuxLoad = 12;  // status word: epilogue waiting for a tile it loads (residual, gate, ...)

enum ElemType { kF16 = 0, kBF16 = 1 };
enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// Two fp32 values -> one packed pair, round to nearest even; `lo` in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t out;
    if constexpr (DT == kF16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(out) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out) : "f"(hi), "f"(lo));
    return out;
}

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (DT == kF16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, long long i) {
    const unsigned short b = static_cast<const unsigned short*>(p)[i];
    if constexpr (DT == kF16) return __half2float(__ushort_as_half(b));
    return __uint_as_float((uint32_t)b << 16);
}

template <int DT>
__device__ __forceinline__ unsigned short pack1(float v) {
    if constexpr (DT == kF16) return __half_as_ushort(__float2half_rn(v));
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Approximations to about 1e-7 of the value; results below 2^-126 are 0.
__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + exp(-y)).  exp(-y) overflows to inf for y below -88, where the
// quotient is 0; __fdividef gives 0 already for a denominator above 2^126.
__device__ __forceinline__ float sigmoid(float y) { return __fdividef(1.0f, 1.0f + __expf(-y)); }

// gelu_tanh(x) = x/2 (1 + tanh z), z = sqrt(2/pi) (x + 0.044715 x^3), is
// x sigmoid(2 z): one exponential, and no cancellation for negative x.
__device__ __forceinline__ float gelu_tanh_2z(float x) {
    return 1.5957691216057308f * x * fmaf(0.044715f * x, x, 1.0f);
}

// The normal distribution's function Phi(x) = (1 + erf(x / sqrt 2)) / 2 and
// exp(-x^2 / 2), by Abramowitz and Stegun's formula 7.1.26: erfc(z) =
// t (a1 + t (a2 + ...)) exp(-z^2) with t = 1 / (1 + p z), off by at most
// 1.5e-7 for z >= 0.  Its exponential is the one the slope needs, and below 0 it is
// the small tail itself, without the cancellation of 1 + erf.
__device__ __forceinline__ float normal_cdf(float x, float& e) {
    const float t = __fdividef(1.0f, fmaf(0.3275911f * 0.70710678118654752f, fabsf(x), 1.0f));
    e = __expf(-0.5f * x * x);
    float q = fmaf(t, 1.061405429f, -1.453152027f);
    q = fmaf(t, q, 1.421413741f);
    q = fmaf(t, q, -0.284496736f);
    q = fmaf(t, q, 0.254829592f);
    const float tail = 0.5f * t * q * e;
    return x < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
    if constexpr (ACT == kActRelu) return x > 0.0f ? x : (x == x ? 0.0f : x);  // NaN stays NaN
    if constexpr (ACT == kActSilu) return __fdividef(x, 1.0f + __expf(-x));
    if constexpr (ACT == kActGelu) {
        float e;
        return x * normal_cdf(x, e);
    }
    if constexpr (ACT == kActGeluTanh) return __fdividef(x, 1.0f + __expf(-gelu_tanh_2z(x)));
    return x;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float x) {
    if constexpr (ACT == kActRelu) return x > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == kActSilu) {
        const float s = sigmoid(x);
        return s * fmaf(x, 1.0f - s, 1.0f);
    }
    if constexpr (ACT == kActGelu) {
        float e;
        const float c = normal_cdf(x, e);
        return fmaf(x * 0.39894228040143268f, e, c);
    }
    if constexpr (ACT == kActGeluTanh) {
        // the slope is 0 or 1 to the last bit beyond |x| = 12; x^3 stays finite (NaN passes through)
        const float c = x > 12.0f ? 12.0f : x < -12.0f ? -12.0f : x;
        const float s = sigmoid(gelu_tanh_2z(c));
        const float dz = 1.5957691216057308f * fmaf(3.0f * 0.044715f * c, c, 1.0f);
        return fmaf(c * s * (1.0f - s), dz, s);
    }
    return 1.0f;
}

// Calls f with the activation as a compile-time tag: chosen once per chunk,
// not per element.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
        case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
        default: f(std::integral_constant<int, kActNone>{}); break;
    }
}

// Instruction descriptor, kind::f16: D fp32, A and B of one 16-bit type, each
// K-major or MN-major.
__host__ __device__ constexpr uint32_t layer_idesc(int dt, bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | ((uint32_t)dt << 7) | ((uint32_t)dt << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One operand's 64-deep K block in shared memory, 128-byte swizzled:
//   K-major   rows of 64 K elements (128 bytes); a K = 16 slice is 32 bytes along the row
//   MN-major  boxes of 64 M (or N) elements x 64 K rows (8 KiB each); a K = 16
//             slice is 16 rows (2 KiB) further down each box
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    return MN ? sw128_desc(saddr, kBoxBytes, 1024) : sw128_desc(saddr, 16, 1024);
}
template <bool MN>
constexpr uint32_t kSliceStep = MN ? (kUmmaK * 128) >> 4 : (kUmmaK * 2) >> 4;  // descriptor units of 16 bytes

__device__ __forceinline__ void st_shared_b16(uint32_t addr, unsigned short v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

__device__ __forceinline__ void ld_shared_f4(uint32_t addr, float& a, float& b, float& c, float& d) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(a), "=f"(b), "=f"(c), "=f"(d)
                 : "r"(addr)
                 : "memory");
}

}  // namespace tcgemm
