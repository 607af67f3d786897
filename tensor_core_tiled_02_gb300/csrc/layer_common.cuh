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
// e = exp(-x^2 / 2).  Phi(-z) = t (c1 + t (c2 + ... t c7)) e for z >= 0 with t = 1 / (1 + p z):
// p and the coefficients minimise the largest relative error, 7.4e-7 over 0 <= z <= 13.5,
// where e ends.  (A formula with an absolute bound will not do: GELU's negative side is the
// tail itself, 6e-12 at x = -7.)  The exponential is the one the slope needs.
constexpr float kTailP = 0.362f;
__host__ __device__ constexpr float tail_coef(int i) {
    constexpr float c[7] = {0.144505310f, 0.142669254f, 0.139541149f, 0.028521731f, 0.177073956f, -0.180350430f, 0.048039397f};
    return c[i];
}

__device__ __forceinline__ float normal_cdf(float x, float& e) {
    const float t = __fdividef(1.0f, fmaf(kTailP, fabsf(x), 1.0f));
    e = __expf(-0.5f * x * x);
    float q = tail_coef(6);
#pragma unroll
    for (int i = 5; i >= 0; --i) q = fmaf(t, q, tail_coef(i));
    const float tail = t * q * e;
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

// ---- two fp32 values at a time -----------------------------------------------------------
// fma.rn.f32x2 and its kin do two in one issue slot: the slope pass is bound by issue
// (GELU's slope is some 25 operations an element one by one) before HBM, and GELU in a
// product's epilogue before the tensor pipe where K is short (4096 tokens, 1024 x 8192: one
// by one 96 us, in pairs 62).

struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 parts(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 both(float c) { return f2(c, c); }
// normal_cdf of two values.
__device__ __forceinline__ F2 normal_cdf2(F2 x, F2& e) {
    F2 ax;
    ax.v = x.v & 0x7FFFFFFF7FFFFFFFull;
    const float2 den = parts(fma2(both(kTailP), ax, both(1.0f)));
    const F2 t = f2(rcp_approx(den.x), rcp_approx(den.y));
    const float2 y = parts(mul2(mul2(x, x), both(-0.72134752044448170f)));
    e = f2(ex2_approx(y.x), ex2_approx(y.y));
    F2 q = both(tail_coef(6));
#pragma unroll
    for (int i = 5; i >= 0; --i) q = fma2(t, q, both(tail_coef(i)));
    const F2 tail = mul2(q, mul2(t, e));
    const float2 lo = parts(tail), hi = parts(fma2(tail, both(-1.0f), both(1.0f))), xs = parts(x);
    return f2(xs.x < 0.0f ? lo.x : hi.x, xs.y < 0.0f ? lo.y : hi.y);
}

// act_value and act_slope of two values.
template <int ACT>
__device__ __forceinline__ F2 act_value2(F2 x) {
    if constexpr (ACT == kActGelu) {
        F2 e;
        return mul2(x, normal_cdf2(x, e));
    }
    const float2 xs = parts(x);
    return f2(act_value<ACT>(xs.x), act_value<ACT>(xs.y));
}
template <int ACT>
__device__ __forceinline__ F2 act_slope2(F2 x) {
    if constexpr (ACT == kActGelu) {
        F2 e;
        const F2 cdf = normal_cdf2(x, e);
        return fma2(mul2(x, both(0.39894228040143268f)), e, cdf);
    }
    const float2 xs = parts(x);
    return f2(act_slope<ACT>(xs.x), act_slope<ACT>(xs.y));
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

// A TMA store writes whole 16-byte pieces: a row that ends inside one would have zeros
// behind it, in what may be another matrix's columns.  So tensor maps of 16-bit outputs end
// at the last whole piece, `n8` = N & ~7 columns, and each lane stores the rest of its row
// from its 16 bytes `piece` in shared memory.
__device__ __forceinline__ void store_tail(uint32_t piece, void* out, long long at, int count) {
    uint32_t w[4];
    ptx::ld_shared_v4(piece, w[0], w[1], w[2], w[3]);
    unsigned short* d = static_cast<unsigned short*>(out) + at;
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < count) d[e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
}

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
