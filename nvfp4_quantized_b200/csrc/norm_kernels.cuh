// norm_kernels.cuh -- layer norm forward and backward.
//
//   mean = sum x / C, rstd = 1/sqrt(sum (x - mean)^2 / C + eps), y = (x - mean) rstd w + b
//   h = (x - mean) rstd, a = dy w:  dx = rstd (a - sum a / C - h sum(a h) / C)
//   dw = sum_r dy h, db = sum_r dy
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"

namespace qt2 {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

constexpr int kNormThreads = 256;

// Sum over the block, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float *sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += sh[i];
    return v;
}

struct NormArgs {
    const void *x, *dy, *w, *b;
    void *y;             // forward: y; backward: dx
    float *mean, *rstd;
    int64_t rows, ldx, lddy, ldy;
    int cols;
    float eps;
    float *part;         // [splits][2][cols]
    int splits;
    void *dw, *db;
};

template <class T, class W>
__global__ void __launch_bounds__(kNormThreads) layernorm_fwd_kernel(const NormArgs a) {
    __shared__ float sh[32];
    const T *x = static_cast<const T *>(a.x) + (int64_t)blockIdx.x * a.ldx;
    T *y = static_cast<T *>(a.y) + (int64_t)blockIdx.x * a.ldy;
    const W *w = static_cast<const W *>(a.w), *b = static_cast<const W *>(a.b);
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) s += to_f32(x[c]);
    const float mean = block_sum(s, sh) / a.cols;
    s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
        const float d = to_f32(x[c]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(block_sum(s, sh) / a.cols + a.eps);
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
        const float h = (to_f32(x[c]) - mean) * rstd;
        const float o = fmaf(h, w ? to_f32(w[c]) : 1.0f, b ? to_f32(b[c]) : 0.0f);
        if (QT2_STORE_OK(y + c, sizeof(T), a.y, ((a.rows - 1) * a.ldy + a.cols) * sizeof(T))) y[c] = from_f32<T>(o);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[blockIdx.x] = mean;
        if (a.rstd) a.rstd[blockIdx.x] = rstd;
    }
}

template <class T, class W>
__global__ void __launch_bounds__(kNormThreads) layernorm_dx_kernel(const NormArgs a) {
    __shared__ float sh[32];
    const T *x = static_cast<const T *>(a.x) + (int64_t)blockIdx.x * a.ldx;
    const T *dy = static_cast<const T *>(a.dy) + (int64_t)blockIdx.x * a.lddy;
    T *dx = static_cast<T *>(a.y) + (int64_t)blockIdx.x * a.ldy;
    const W *w = static_cast<const W *>(a.w);
    const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
    float s = 0.0f, q = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
        const float h = (to_f32(x[c]) - mean) * rstd, g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.0f);
        s += g;
        q = fmaf(g, h, q);
    }
    s = block_sum(s, sh) / a.cols;
    q = block_sum(q, sh) / a.cols;
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
        const float h = (to_f32(x[c]) - mean) * rstd, g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.0f);
        if (QT2_STORE_OK(dx + c, sizeof(T), a.y, ((a.rows - 1) * a.ldy + a.cols) * sizeof(T)))
            dx[c] = from_f32<T>(rstd * (g - s - h * q));
    }
}

// Partial sums of dw and db over rows split, split + splits, ...: one thread a column.
template <class T>
__global__ void __launch_bounds__(kNormThreads) layernorm_dw_part_kernel(const NormArgs a) {
    const int c = blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < a.rows; r += a.splits) {
        const float g = to_f32(static_cast<const T *>(a.dy)[r * a.lddy + c]);
        db += g;
        dw = fmaf(g, (to_f32(static_cast<const T *>(a.x)[r * a.ldx + c]) - a.mean[r]) * a.rstd[r], dw);
    }
    a.part[((int64_t)blockIdx.y * 2) * a.cols + c] = dw;
    a.part[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = db;
}

template <class W>
__global__ void __launch_bounds__(kNormThreads) layernorm_dw_kernel(const NormArgs a) {
    const int c = blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (int i = 0; i < a.splits; ++i) {
        dw += a.part[((int64_t)i * 2) * a.cols + c];
        db += a.part[((int64_t)i * 2 + 1) * a.cols + c];
    }
    if (a.dw && QT2_STORE_OK(static_cast<W *>(a.dw) + c, sizeof(W), a.dw, a.cols * sizeof(W)))
        static_cast<W *>(a.dw)[c] = from_f32<W>(dw);
    if (a.db && QT2_STORE_OK(static_cast<W *>(a.db) + c, sizeof(W), a.db, a.cols * sizeof(W)))
        static_cast<W *>(a.db)[c] = from_f32<W>(db);
}

}  // namespace qt2
