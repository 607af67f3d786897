// The global norm of many gradients and their clipping.
//
//   norm = sqrt(sum over all tensors and entries of g^2)
//   g    = g min(1, max_norm / (norm + eps))
//
// Bound by memory: the norm has to be whole before the first entry can be
// scaled, so the gradients are read twice (the second time in the opposite
// order, so that what the norm pass read last is found in L2) and written
// once.  The tensors' table travels in the kernel's parameters; a block
// takes chunks of up to kClipMostChunk entries of one tensor.  Squares are summed in fp32:
// 64 terms per thread and chunk, then chunk by chunk, then pairwise over the
// threads and blocks, in a fixed order (fp64 runs at a small fraction of fp32's rate
// on this GPU).  Norms between 1e-19 and 1e19 are what fp32 squares can hold.
//
// 700 M bf16 entries in 290 tensors: 781 us, 4.88 GB over the three passes at 6.2
// TB/s; 400,000 fp32 entries in 24 tensors: 4.7 us, two launches.
#pragma once

#include "layer_common.cuh"

namespace tcgemm {

constexpr int kClipThreads = 256;
constexpr int kClipMostChunk = 32768;  // entries; fewer where the tensors are few and small, so that
constexpr int kClipLeastChunk = 2048;  // every SM has some (400,000 entries: 9.1 us in 32768s, 4.7 in 2048s)
constexpr int kClipF32 = 2;         // ElemType's continuation

struct ClipEntry {
    const void* src;
    void* dst;
    long long count_type;           // entries * 4 + type
};

template <int CAP>
struct ClipTable {
    int tensors, chunks, chunk;     // chunk: entries
    int first[CAP];                 // first chunk of each tensor
    ClipEntry e[CAP];
};

template <int CAP>
__device__ __forceinline__ int clip_find(const ClipTable<CAP>& t, int chunk) {
    int lo = 0, hi = t.tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int TY>
__device__ __forceinline__ float clip_load(const void* p, int i) {
    if constexpr (TY == kClipF32) return static_cast<const float*>(p)[i];
    else return load1<TY>(p, i);
}
template <int TY>
__device__ __forceinline__ void clip_store(void* p, int i, float v) {
    if constexpr (TY == kClipF32) static_cast<float*>(p)[i] = v;
    else static_cast<unsigned short*>(p)[i] = pack1<TY>(v);
}
template <int TY>
constexpr int kClipBytes = TY == kClipF32 ? 4 : 2;

// Entries before the first 16-byte boundary (pointers are aligned to their type).
template <int TY>
__device__ __forceinline__ int clip_head(const void* p, int n) {
    const int h = (int)((16 - ((uintptr_t)p & 15)) & 15) / kClipBytes<TY>;
    return h < n ? h : n;
}

template <int TY>
__device__ __forceinline__ float clip_squares(const void* src, int n) {
    constexpr int V = 16 / kClipBytes<TY>;
    const int head = clip_head<TY>(src, n);
    const int vecs = (n - head) / V;
    const char* body = static_cast<const char*>(src) + head * kClipBytes<TY>;
    float s0 = 0.0f, s1 = 0.0f;
    if ((int)threadIdx.x < head) {
        const float v = clip_load<TY>(src, threadIdx.x);
        s0 = v * v;
    }
    const int tail = head + vecs * V + (int)threadIdx.x;
    if (tail < n) {
        const float v = clip_load<TY>(src, tail);
        s1 = v * v;
    }
#pragma unroll 8
    for (int i = threadIdx.x; i < vecs; i += kClipThreads) {
        const uint4 w = reinterpret_cast<const uint4*>(body)[i];
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (TY == kClipF32) {
                const float v = __uint_as_float(ws[e]);
                if (e & 1) s1 = fmaf(v, v, s1); else s0 = fmaf(v, v, s0);
            } else {
                const float2 f = unpack2<TY>(ws[e]);
                s0 = fmaf(f.x, f.x, s0);
                s1 = fmaf(f.y, f.y, s1);
            }
        }
    }
    return s0 + s1;
}

// The sum of every thread's v, in a fixed order; all threads get it.
__device__ __forceinline__ float clip_block_sum(float v, float* scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kClipThreads / 32; ++i) v += scratch[i];
    return v;
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads)
    clip_norm_kernel(const __grid_constant__ ClipTable<CAP> t, float* partial) {
    __shared__ float sums[kClipThreads / 32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float total = 0.0f;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int k = clip_find(t, c);
        const ClipEntry& e = t.e[k];
        const long long at = (long long)(c - t.first[k]) * t.chunk;
        const long long left = (e.count_type >> 2) - at;
        const int n = (int)(left < t.chunk ? left : t.chunk);
        const int ty = (int)(e.count_type & 3);
        const char* src = static_cast<const char*>(e.src) + at * (ty == kClipF32 ? 4 : 2);
        total += (ty == kClipF32 ? clip_squares<kClipF32>(src, n)
                          : ty == kBF16 ? clip_squares<kBF16>(src, n) : clip_squares<kF16>(src, n));
    }
    total = clip_block_sum(total, sums);
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

template <int TY>
__device__ __forceinline__ void clip_scale(const void* src, void* dst, int n, float coef) {
    constexpr int V = 16 / kClipBytes<TY>;
    if ((((uintptr_t)src ^ (uintptr_t)dst) & 15) != 0) {  // no common 16-byte boundary
        for (int i = threadIdx.x; i < n; i += kClipThreads) clip_store<TY>(dst, i, clip_load<TY>(src, i) * coef);
        return;
    }
    const int head = clip_head<TY>(src, n);
    const int vecs = (n - head) / V;
    if ((int)threadIdx.x < head) clip_store<TY>(dst, threadIdx.x, clip_load<TY>(src, threadIdx.x) * coef);
    const int tail = head + vecs * V + (int)threadIdx.x;
    if (tail < n) clip_store<TY>(dst, tail, clip_load<TY>(src, tail) * coef);
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(src) + head * kClipBytes<TY>);
    uint4* d = reinterpret_cast<uint4*>(static_cast<char*>(dst) + head * kClipBytes<TY>);
    constexpr int U = 8;
    for (int i0 = threadIdx.x; i0 < vecs; i0 += kClipThreads * U) {
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * kClipThreads < vecs) w[u] = s[i0 + u * kClipThreads];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * kClipThreads >= vecs) break;
            uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (TY == kClipF32) {
                    ws[e] = __float_as_uint(__uint_as_float(ws[e]) * coef);
                } else {
                    const float2 f = unpack2<TY>(ws[e]);
                    ws[e] = pack2<TY>(f.x * coef, f.y * coef);
                }
            }
            d[i0 + u * kClipThreads] = make_uint4(ws[0], ws[1], ws[2], ws[3]);
        }
    }
}

// Every block sums the partials itself, in order (a few KiB from L2).
template <int CAP>
__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipTable<CAP> t, const float* partial, int parts, float max_norm,
                      float eps, float* norm_out) {
    __shared__ float sums[kClipThreads / 32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    float total = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < parts; i += kClipThreads) total += partial[i];
    const float norm = sqrtf(clip_block_sum(total, sums));
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out != nullptr) *norm_out = norm;
    const float c = max_norm / (norm + eps);
    const float coef = c < 1.0f ? c : c == c ? 1.0f : c;  // a NaN norm makes every entry NaN
    for (int k = blockIdx.x; k < t.chunks; k += gridDim.x) {
        const int ch = t.chunks - 1 - k;
        const int i = clip_find(t, ch);
        const ClipEntry& e = t.e[i];
        // in place and nothing to clip: the entries stay as they are
        if (coef == 1.0f && e.src == e.dst) continue;
        const long long at = (long long)(ch - t.first[i]) * t.chunk;
        const long long left = (e.count_type >> 2) - at;
        const int n = (int)(left < t.chunk ? left : t.chunk);
        const int ty = (int)(e.count_type & 3);
        const char* src = static_cast<const char*>(e.src) + at * (ty == kClipF32 ? 4 : 2);
        char* dst = static_cast<char*>(e.dst) + at * (ty == kClipF32 ? 4 : 2);
        if (ty == kClipF32) clip_scale<kClipF32>(src, dst, n, coef);
        else if (ty == kBF16) clip_scale<kBF16>(src, dst, n, coef);
        else clip_scale<kF16>(src, dst, n, coef);
    }
}

}  // namespace tcgemm
