// rope_kernels.cuh -- the norm of queries and keys for each head with the position rotation, and its
// backward pass.
//
//   r = 1 / sqrt(sum x^2 / D + eps), n = x r, a = n w, y = a turned by its position's angles   (forward)
//   b = dy turned back, dw = sum over tokens and heads of b n,
//   dx = r (b w - n sum(b w n) / D)                                                            (backward)
//
// A row is one head of one token.  The members of a rotated pair, (i, i + R/2) or (2i, 2i + 1), belong to
// one lane: a lane's slot is two chunks of 4 elements, R/2 apart or next to each other, with the same 4
// angles either way.  No element passes between lanes; only the row's one or two sums do, by shuffles.
// G lanes share a row (N slots each), and a group takes U rows that follow one another, whose loads are
// all issued before the first is used.  Backward recomputes r from x, which it reads anyway.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"
#include "vec_device.cuh"

namespace qt2 {

constexpr int kQkThreads = 256;

struct QkArgs {
    const void *x, *dy;
    void *y;                       // y, or dx (may be null)
    const void *w[2];              // of queries and keys; null: ones
    void *dw[2];
    const int64_t *pos;            // null: the token's number
    const float *cos, *sin;        // [P][R / 2]
    int64_t P, T;
    int heads[2], D, R;
    int64_t ldx, hsx, ldy, hsy, lddy, hsdy;   // between tokens, between heads
    int pairs, w_f32;
    float eps;
    float *part;                   // [blocks][2][D], or null
    int parts;
};

// Four elements in memory as they are loaded.
template <class T>
struct QkChunk;
template <>
struct QkChunk<__nv_bfloat16> {
    uint2 r;
    __device__ __forceinline__ void get(float *v) const {
        v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
    }
    __device__ __forceinline__ void set(const float *v) { r = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])); }
};
template <>
struct QkChunk<float> {
    float4 r;
    __device__ __forceinline__ void get(float *v) const { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
    __device__ __forceinline__ void set(const float *v) { r = make_float4(v[0], v[1], v[2], v[3]); }
};

// Where a slot's two chunks are in a head, and whether they are rotated (by angles 4 s ... 4 s + 3).
struct QkSlot {
    int c0, c1;
    bool live, turned;
};
__device__ __forceinline__ QkSlot qk_slot(const QkArgs &a, int s) {
    QkSlot q;
    q.live = s < a.D / 8;
    q.turned = s < a.R / 8;
    if (a.pairs) {
        q.c0 = 8 * s;
        q.c1 = 8 * s + 4;
    } else if (q.turned) {
        q.c0 = 4 * s;
        q.c1 = a.R / 2 + 4 * s;
    } else {
        q.c0 = a.R + 4 * (s - a.R / 8);
        q.c1 = q.c0 + (a.D - a.R) / 2;
    }
    return q;
}

template <class T>
__device__ __forceinline__ void qk_load(const void *base, int64_t at, const QkSlot &q, QkChunk<T> (&c)[2]) {
    const T *p = static_cast<const T *>(base) + at;
    c[0] = *reinterpret_cast<const QkChunk<T> *>(p + q.c0);
    c[1] = *reinterpret_cast<const QkChunk<T> *>(p + q.c1);
}
template <class T>
__device__ __forceinline__ void qk_store(const QkArgs &a, int64_t at, const QkSlot &q, const float (&v)[8]) {
    T *const base = static_cast<T *>(a.y);
    const int64_t size = ((a.T - 1) * a.ldy + (a.heads[0] + a.heads[1] - 1) * a.hsy + a.D) * (int64_t)sizeof(T);
    QkChunk<T> c[2];
    c[0].set(v);
    c[1].set(v + 4);
    if (QT2_STORE_OK(base + at + q.c0, 4 * sizeof(T), base, size)) *reinterpret_cast<QkChunk<T> *>(base + at + q.c0) = c[0];
    if (QT2_STORE_OK(base + at + q.c1, 4 * sizeof(T), base, size)) *reinterpret_cast<QkChunk<T> *>(base + at + q.c1) = c[1];
}
__device__ __forceinline__ void qk_weight(const QkArgs &a, int kind, const QkSlot &q, float (&w)[8]) {
    const void *p = a.w[kind];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    if (!p || !q.live) return;
    if (a.w_f32) {
        QkChunk<float> c[2];
        qk_load<float>(p, 0, q, c);
        c[0].get(w);
        c[1].get(w + 4);
    } else {
        QkChunk<__nv_bfloat16> c[2];
        qk_load<__nv_bfloat16>(p, 0, q, c);
        c[0].get(w);
        c[1].get(w + 4);
    }
}
__device__ __forceinline__ void qk_angles(const QkArgs &a, int64_t pos, const QkSlot &q, int s, float4 &c, float4 &d) {
    c = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    d = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!q.turned || (uint64_t)pos >= (uint64_t)a.P) return;
    const int64_t at = pos * (a.R / 2) + 4 * s;
    c = *reinterpret_cast<const float4 *>(a.cos + at);
    d = *reinterpret_cast<const float4 *>(a.sin + at);
}
// Pair p is (v[p], v[4 + p]), or (v[2 p], v[2 p + 1]).
__device__ __forceinline__ void qk_turn(float (&v)[8], const float4 &c4, const float4 &s4, int pairs, float sign) {
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x * sign, s4.y * sign, s4.z * sign, s4.w * sign};
    if (pairs) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float x = v[2 * p], y = v[2 * p + 1];
            v[2 * p] = x * c[p] - y * s[p];
            v[2 * p + 1] = y * c[p] + x * s[p];
        }
    } else {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float x = v[p], y = v[4 + p];
            v[p] = x * c[p] - y * s[p];
            v[4 + p] = y * c[p] + x * s[p];
        }
    }
}

// U rows of a group: rows [row, row + U) of a kind's T x heads, token by token.
template <int U>
struct QkRows {
    int64_t t[U], pos[U];
    int h[U];
    bool live[U];
};
template <int U>
__device__ __forceinline__ void qk_rows(const QkArgs &a, int kind, int64_t row, QkRows<U> &q) {
    const int H = a.heads[kind];
    const int64_t n = a.T * H;
    int64_t t = row < n ? row / H : 0;
    int h = (int)(row < n ? row - t * H : 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        q.live[u] = row + u < n;
        q.t[u] = q.live[u] ? t : 0;
        q.h[u] = q.live[u] ? h + (kind ? a.heads[0] : 0) : 0;
        if (++h == H) h = 0, ++t;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        q.pos[u] = a.R == 0 ? 0 : a.pos ? a.pos[q.t[u]] : q.t[u];
        if (a.R && q.live[u] && (uint64_t)q.pos[u] >= (uint64_t)a.P) set_device_error(QT2_ERR_INVALID_ARG);
    }
}

template <class T, int G, int N, int U>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_fwd_kernel(const __grid_constant__ QkArgs a) {
    constexpr int kRows = 32 / G * U;   // of a warp
    grid_dependency();
    const int lane = threadIdx.x & 31, g = lane % G;
    const float inv_d = 1.0f / (float)a.D;
    const int64_t items[2] = {(a.T * a.heads[0] + kRows - 1) / kRows, (a.T * a.heads[1] + kRows - 1) / kRows};
    int64_t item = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5);
    const int kind = item >= items[0];
    if (kind) item -= items[0];
    if (item >= items[kind]) return;
    QkRows<U> rows;
    qk_rows<U>(a, kind, item * kRows + lane / G * U, rows);
    QkSlot slot[N];
    QkChunk<T> raw[U][N][2] = {};
    float4 c[U][N], s[U][N];
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i] = qk_slot(a, g + i * G);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (slot[i].live && rows.live[u]) qk_load<T>(a.x, rows.t[u] * a.ldx + rows.h[u] * a.hsx, slot[i], raw[u][i]);
    float w[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) qk_weight(a, kind, slot[i], w[i]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i) qk_angles(a, rows.pos[u], slot[i], g + i * G, c[u][i], s[u][i]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[N][8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            raw[u][i][0].get(v[i]);
            raw[u][i][1].get(v[i] + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(v[i][e], v[i][e], sum);
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float r = rsqrtf(fmaf(sum, inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * r * w[i][e];
            qk_turn(v[i], c[u][i], s[u][i], a.pairs, 1.0f);
            if (slot[i].live && rows.live[u]) qk_store<T>(a, rows.t[u] * a.ldy + rows.h[u] * a.hsy, slot[i], v[i]);
        }
    }
}

// part[block][kind][D]: the block's share of dw.
template <class T, int G, int N, int U>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_bwd_kernel(const __grid_constant__ QkArgs a) {
    constexpr int kRows = 32 / G * U, kWarps = kQkThreads / 32;
    extern __shared__ float sums[];   // [kWarps][D]
    grid_dependency();
    const int lane = threadIdx.x & 31, g = lane % G, warp = threadIdx.x >> 5;
    const float inv_d = 1.0f / (float)a.D;
    QkSlot slot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i] = qk_slot(a, g + i * G);
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        float w[N][8], acc[N][8];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            qk_weight(a, kind, slot[i], w[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
        }
        const int64_t items = (a.T * a.heads[kind] + kRows - 1) / kRows;
#pragma unroll 1
        for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < items; item += (int64_t)gridDim.x * kWarps) {
            QkRows<U> rows;
            qk_rows<U>(a, kind, item * kRows + lane / G * U, rows);
            QkChunk<T> raw[U][N][2] = {}, up[U][N][2] = {};   // zeros where no row or slot is
            float4 c[U][N], s[U][N];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (slot[i].live && rows.live[u]) {
                        qk_load<T>(a.x, rows.t[u] * a.ldx + rows.h[u] * a.hsx, slot[i], raw[u][i]);
                        qk_load<T>(a.dy, rows.t[u] * a.lddy + rows.h[u] * a.hsdy, slot[i], up[u][i]);
                    }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < N; ++i) qk_angles(a, rows.pos[u], slot[i], g + i * G, c[u][i], s[u][i]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[N][8], b[N][8], sum = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    raw[u][i][0].get(v[i]);
                    raw[u][i][1].get(v[i] + 4);
                    up[u][i][0].get(b[i]);
                    up[u][i][1].get(b[i] + 4);
                    qk_turn(b[i], c[u][i], s[u][i], a.pairs, -1.0f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sum = fmaf(v[i][e], v[i][e], sum);
                        dot = fmaf(b[i][e] * w[i][e], v[i][e], dot);
                    }
                }
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) {
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
                }
                const float r = rsqrtf(fmaf(sum, inv_d, a.eps));
                const float mean = dot * r * inv_d;   // of b w n
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float n = v[i][e] * r;
                        d[e] = r * fmaf(-n, mean, b[i][e] * w[i][e]);
                        if (rows.live[u]) acc[i][e] = fmaf(b[i][e], n, acc[i][e]);   // r may be inf where no row is
                    }
                    if (a.y && slot[i].live && rows.live[u])
                        qk_store<T>(a, rows.t[u] * a.ldy + rows.h[u] * a.hsy, slot[i], d);
                }
            }
        }
        if (!a.part) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int o = G; o < 32; o <<= 1) acc[i][e] += __shfl_xor_sync(0xFFFFFFFFu, acc[i][e], o);
            if (lane < G && slot[i].live) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[warp * a.D + (e < 4 ? slot[i].c0 + e : slot[i].c1 + e - 4)] = acc[i][e];
            }
        }
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += kQkThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) sum += sums[k * a.D + d];
            put(a.part, ((int64_t)blockIdx.x * 2 + kind) * a.D + d, (int64_t)a.parts * 2 * a.D, sum);
        }
        __syncthreads();
    }
}

// dw of queries (blockIdx.y = 0) and keys: the blocks' shares in their order, 32 columns a block.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const __grid_constant__ QkArgs a) {
    __shared__ float sums[32][33];
    grid_dependency();
    const int kind = blockIdx.y, d = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    if (!a.dw[kind]) return;
    float sum = 0.0f;
    if (d < a.D)
        for (int p = k; p < a.parts; p += 32) sum += a.part[((int64_t)p * 2 + kind) * a.D + d];
    sums[k][threadIdx.x & 31] = sum;
    __syncthreads();
    sum = sums[threadIdx.x & 31][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const int out = blockIdx.x * 32 + k;
    if ((threadIdx.x & 31) != 0 || out >= a.D) return;
    if (a.w_f32)
        put(static_cast<float *>(a.dw[kind]), out, a.D, sum);
    else
        put(static_cast<__nv_bfloat16 *>(a.dw[kind]), out, a.D, __float2bfloat16_rn(sum));
}

}  // namespace qt2
