// The linear layer on microscaled operands, element by element.
#pragma once

#include "mx_common.cuh"

namespace tcgemm {

struct MxLinearParams {
    const uint8_t *x, *x_scale, *w, *w_scale;
    const void *bias, *residual;
    void* y;
    long long ldx, ldw, ldr, ldy;
    int tokens, n, blocks;
    int act;
};

// A thread an element of y.
template <int DT, int FMT>
__global__ void __launch_bounds__(256) mx_linear_simple_kernel(const MxLinearParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const long long at = blockIdx.x * 256ll + threadIdx.x;
    const long long t = at / p.n, c = at % p.n;
    if (t >= p.tokens) return;
    const int k_tiles = (p.blocks + 3) >> 2;
    float sum = 0.0f;
    for (int b = 0; b < p.blocks; ++b) {
        const float scale = mx_scale_value(p.x_scale[mx_scale_word(t, b >> 2, k_tiles) + (b & 3)]) *
                            mx_scale_value(p.w_scale[mx_scale_word(c, b >> 2, k_tiles) + (b & 3)]);
        constexpr int kBytes = mx_block_bytes(FMT);
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            auto eight = [&](const uint8_t* d, float(&f)[8]) {
                uint2 q = make_uint2(*reinterpret_cast<const uint32_t*>(d), 0u);
                if constexpr (FMT == kE4M3) q.y = *reinterpret_cast<const uint32_t*>(d + 4);
                mx_unpack8<FMT>(q, 1.0f, f);
            };
            float a[8], w[8];
            eight(p.x + t * p.ldx + b * kBytes + i * (kBytes / 4), a);
            eight(p.w + c * p.ldw + b * kBytes + i * (kBytes / 4), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) part = fmaf(a[e], w[e], part);
        }
        sum = fmaf(part, scale, sum);
    }
    if (p.bias != nullptr) sum += load1<DT>(p.bias, c);
    if (p.act != kActNone) with_act(p.act, [&](auto tag) { sum = act_value<decltype(tag)::value>(sum); });
    if (p.residual != nullptr) sum += load1<DT>(p.residual, t * p.ldr + c);
    static_cast<unsigned short*>(p.y)[t * p.ldy + c] = pack1<DT>(sum);
}

}  // namespace tcgemm
