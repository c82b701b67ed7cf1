// grad_kernels.cuh -- the global norm of a list of gradients, and clipping by it.
//
//   norm = sqrt(sum_i sum_j g_ij^2),  out = g min(1, max_norm / (norm + 1e-6))
//
// Both are streams over HBM: one read for the norm, one read and one write for the clipping (411M fp32
// gradients: 0.73 to 0.75 ms for the two, 6.6 to 6.8 TB/s, in place or not).  The list travels in the kernel's parameters (no copy to
// the device, nothing that a captured graph could find changed).  Tensors are cut into chunks of
// 16-byte vectors, counted from the aligned address at or below the tensor's first element; a thread
// has kGradVecs of them in flight.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"

namespace qt2 {

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;
constexpr int kGradChunk = kGradThreads * kGradVecs;   // vectors a block takes at a time: 32 KB
constexpr int kGradSmall = 32, kGradMiddle = 256, kGradLarge = 1024;   // tensors a launch's parameters hold

template <int N>
struct GradTable {
    const void *grad[N];
    void *out[N];
    int64_t numel[N];
    int32_t first[N + 1];      // chunks before tensor i; first[count] is their sum
    uint32_t f32[N / 32];      // bit i: tensor i is fp32
    int count;
};

// One chunk of a tensor: its vectors [lo, hi) from the aligned address `base` on, of which elements
// [head, end) are the tensor's (counted from base).
struct GradChunk {
    const uint8_t *base;
    int64_t lo, hi, head, end;
    int tensor;
    bool f32;
};

template <int N>
__device__ __forceinline__ GradChunk grad_chunk(const GradTable<N> &t, int chunk) {
    int k = 0, top = t.count - 1;
    while (k < top) {
        const int mid = (k + top + 1) >> 1;
        if (t.first[mid] <= chunk)
            k = mid;
        else
            top = mid - 1;
    }
    GradChunk c;
    c.tensor = k;
    c.f32 = (t.f32[k >> 5] >> (k & 31)) & 1;
    const uintptr_t p = reinterpret_cast<uintptr_t>(t.grad[k]);
    c.base = reinterpret_cast<const uint8_t *>(p & ~uintptr_t(15));
    const int shift = c.f32 ? 2 : 1;
    c.head = (int64_t)(p & 15) >> shift;
    c.end = c.head + t.numel[k];
    c.lo = (int64_t)(chunk - t.first[k]) * kGradChunk;
    c.hi = min(c.lo + kGradChunk, (c.end + (16 >> shift) - 1) >> (4 - shift));
    return c;
}

// The fp32 values of a vector; elements that are not the tensor's are zero.
__device__ __forceinline__ void grad_values(const uint4 &r, const GradChunk &c, int64_t vec, float (&v)[8]) {
    if (c.f32) {
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
        v[4] = v[5] = v[6] = v[7] = 0.0f;
    } else {
        v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
        v[4] = bf16_lo(r.z); v[5] = bf16_hi(r.z); v[6] = bf16_lo(r.w); v[7] = bf16_hi(r.w);
    }
    const int n = c.f32 ? 4 : 8;
    const int64_t at = vec * n;
    if (at < c.head || at + n > c.end) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (at + e < c.head || at + e >= c.end) v[e] = 0.0f;
    }
}

// The vector's sum of squares.  In fp32 where that loses nothing: from 2^-80 up squares that underflow
// are 2^-43 of it at most, and up to 2^120 none overflowed; else (also zeros, inf and NaN) in fp64.
__device__ __forceinline__ double grad_squares(const float (&v)[8]) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
    if (s >= 0x1p-80f && s <= 0x1p120f) return (double)s;
    float any = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) any = fmaxf(any, fabsf(v[e]));   // 0 for a vector of NaNs, whose s is NaN
    if (any == 0.0f) return (double)s;
    double d = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) d += (double)v[e] * (double)v[e];
    return d;
}

__device__ __forceinline__ double grad_block_sum(double sum) {
    __shared__ double sh[kGradThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kGradThreads / 32; ++i) sum += sh[i];
    return sum;
}

// part[blockIdx.x] = the sum of squares of the block's chunks, or (norm given: the blocks are one
// cluster, and the launch the only one) the norm itself.
template <int N>
__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const __grid_constant__ GradTable<N> t, double *part,
                                                                 float *norm) {
    grid_dependency();
    double sum = 0.0;
    for (int k = blockIdx.x; k < t.first[t.count]; k += gridDim.x) {
        const GradChunk c = grad_chunk(t, k);
        uint4 r[kGradVecs];
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const int64_t v = c.lo + threadIdx.x + i * kGradThreads;
            r[i] = v < c.hi ? *(reinterpret_cast<const uint4 *>(c.base) + v) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            float f[8];
            grad_values(r[i], c, c.lo + threadIdx.x + i * kGradThreads, f);
            sum += grad_squares(f);
        }
    }
    sum = grad_block_sum(sum);
    if (!norm) {
        if (threadIdx.x == 0) put(part, (int64_t)blockIdx.x, (int64_t)gridDim.x, sum);
        return;
    }
    __shared__ double mine;
    if (threadIdx.x == 0) mine = sum;
    cluster_sync_all();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        sum = 0.0;
        for (uint32_t q = 0; q < gridDim.x; ++q) {
            const uint32_t at = mapa_shared(smem_u32(&mine), q);
            sum += __hiloint2double((int)ld_shared_cluster_u32(at + 4), (int)ld_shared_cluster_u32(at));
        }
        put(norm, 0, 1, (float)sqrt(sum));
    }
    cluster_sync_all();   // no block leaves while the first reads its sum
}

__global__ void __launch_bounds__(kGradThreads) grad_norm_end_kernel(const double *part, int n, float *norm) {
    grid_dependency();
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kGradThreads) sum += part[i];
    sum = grad_block_sum(sum);
    if (threadIdx.x == 0) put(norm, 0, 1, (float)sqrt(sum));
}

// The chunks from the last to the first: what the norm's pass read last is still in L2.
template <int N>
__global__ void __launch_bounds__(kGradThreads, 3) grad_clip_kernel(const __grid_constant__ GradTable<N> t,
                                                                 const float *norm, float max_norm) {
    grid_dependency();
    const float q = max_norm / (*norm + 1e-6f), f = q > 1.0f ? 1.0f : q;   // a NaN stays
    for (int k = t.first[t.count] - 1 - (int)blockIdx.x; k >= 0; k -= gridDim.x) {
        const GradChunk c = grad_chunk(t, k);
        if (f == 1.0f && t.out[c.tensor] == t.grad[c.tensor]) continue;
        // the output's address that belongs to `base`
        uint8_t *const out = static_cast<uint8_t *>(t.out[c.tensor]) - (c.head << (c.f32 ? 2 : 1));
        const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        uint4 r[kGradVecs];
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const int64_t v = c.lo + threadIdx.x + i * kGradThreads;
            r[i] = v < c.hi ? *(reinterpret_cast<const uint4 *>(c.base) + v) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const int64_t v = c.lo + threadIdx.x + i * kGradThreads;
            if (v >= c.hi) continue;
            const int n = c.f32 ? 4 : 8;
            const int64_t at = v * n;
            float x[8];
            grad_values(r[i], c, v, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= f;
            const int64_t size = (c.end - c.head) * (c.f32 ? 4 : 2);
            if (same && at >= c.head && at + n <= c.end) {
                uint4 w;
                if (c.f32) {
                    w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                   __float_as_uint(x[3]));
                } else {
                    uint32_t p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                        p[e] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                    w = make_uint4(p[0], p[1], p[2], p[3]);
                }
                if (QT2_STORE_OK(out + v * 16, 16, t.out[c.tensor], size)) *reinterpret_cast<uint4 *>(out + v * 16) = w;
                continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e >= n || at + e < c.head || at + e >= c.end) continue;
                if (c.f32) {
                    float *p = reinterpret_cast<float *>(out) + at + e;
                    if (QT2_STORE_OK(p, 4, t.out[c.tensor], size)) *p = x[e];
                } else {
                    __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(out) + at + e;
                    if (QT2_STORE_OK(p, 2, t.out[c.tensor], size)) *p = __float2bfloat16_rn(x[e]);
                }
            }
        }
    }
}

}  // namespace qt2
