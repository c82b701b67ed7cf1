// grad_kernels.cuh -- the global norm of a list of gradients, and clipping by it.
//
//   norm = sqrt(sum_i sum_j g_ij^2),  out = g min(1, max_norm / (norm + 1e-6))
//
// The list travels in the kernel's parameters (no copy to the device, nothing that a captured
// graph could find changed); tensors are cut into chunks that the blocks take in turn.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"

namespace qt2 {

constexpr int kGradThreads = 256;
constexpr int kGradChunk = 8192;        // elements a block takes at a time
constexpr int kGradTable = 128;         // tensors a launch takes

struct GradTable {
    const void *grad[kGradTable];
    void *out[kGradTable];
    int64_t numel[kGradTable];
    int64_t first[kGradTable + 1];      // chunks before tensor i; first[count] is their sum
    uint32_t f32[kGradTable / 32];      // bit i: tensor i is fp32
    int count;
};

__device__ __forceinline__ int grad_find(const GradTable &t, int64_t chunk) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float grad_load(const void *p, int64_t i, bool f32) {
    return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradTable t, double *part) {
    __shared__ double sh[kGradThreads / 32];
    double sum = 0.0;
    const int64_t chunks = t.first[t.count];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int k = grad_find(t, c);
        const int64_t lo = (c - t.first[k]) * kGradChunk, hi = min(t.numel[k], lo + kGradChunk);
        const bool f32 = (t.f32[k >> 5] >> (k & 31)) & 1;
        for (int64_t i = lo + threadIdx.x; i < hi; i += kGradThreads) {
            const double g = grad_load(t.grad[k], i, f32);
            sum += g * g;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kGradThreads / 32; ++i) sum += sh[i];
        part[blockIdx.x] = sum;
    }
}

__global__ void __launch_bounds__(kGradThreads) grad_norm_end_kernel(const double *part, int n, float *norm) {
    __shared__ double sh[kGradThreads / 32];
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kGradThreads) sum += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kGradThreads / 32; ++i) sum += sh[i];
        *norm = (float)sqrt(sum);
    }
}

__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(const __grid_constant__ GradTable t,
                                                                 const float *norm, float max_norm) {
    const float r = max_norm / (*norm + 1e-6f), f = r > 1.0f ? 1.0f : r;   // a NaN stays
    const int64_t chunks = t.first[t.count];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int k = grad_find(t, c);
        if (f == 1.0f && t.out[k] == t.grad[k]) continue;
        const int64_t lo = (c - t.first[k]) * kGradChunk, hi = min(t.numel[k], lo + kGradChunk);
        const bool f32 = (t.f32[k >> 5] >> (k & 31)) & 1;
        for (int64_t i = lo + threadIdx.x; i < hi; i += kGradThreads) {
            const float g = grad_load(t.grad[k], i, f32) * f;
            if (!QT2_STORE_OK(static_cast<uint8_t *>(t.out[k]) + i * (f32 ? 4 : 2), f32 ? 4 : 2, t.out[k],
                              t.numel[k] * (f32 ? 4 : 2)))
                continue;
            if (f32)
                static_cast<float *>(t.out[k])[i] = g;
            else
                static_cast<__nv_bfloat16 *>(t.out[k])[i] = __float2bfloat16_rn(g);
        }
    }
}

}  // namespace qt2
