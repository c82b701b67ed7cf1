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
// G lanes share a row (N slots each), and a group takes U heads of a token, which share their angles; their
// loads are all issued before the first is used.  Backward recomputes r from x, which it reads anyway.
//
// A stream over HBM that instructions hold back: 17 an element forward (issue 68%, 5.1 TB/s: 32768 x 16+16 x 128 bf16
// 105 to 108 us, 83 for its bytes), 21 backward (54% with 16 warps an SM, 5.0 TB/s: 159 to 164 us, 124 for its bytes).
// Four heads a group share the angles' loads and the index arithmetic (one head: 168 and 282 us); conditional
// loads, or the next unit's ahead of this one's work, were slower (147; 202 to 270 us).  fp32, half the tokens: 92 and
// 138 us (5.9 TB/s).
#pragma once

#include <cuda_bf16.h>
#include <type_traits>

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
    uint32_t ldx, hsx, ldy, hsy, lddy, hsdy;   // between tokens, between heads
    int w_f32;
    float eps;
    float *part;                   // [blocks][2][D], or null
    int parts;
};

// A slot's eight elements as they lie in memory: two chunks of four.
template <class T>
struct QkRaw;
template <>
struct QkRaw<__nv_bfloat16> {
    uint2 c[2];
};
template <>
struct QkRaw<float> {
    float4 c[2];
};
// The same as the first (x) and the second members (y) of four pairs.
struct QkPairs {
    uint64_t x[2], y[2];
};
template <bool PAIRS>
__device__ __forceinline__ QkPairs qk_get(const QkRaw<__nv_bfloat16> &r) {
    const uint2 a = r.c[0], b = r.c[1];
    if constexpr (PAIRS)
        return {{f2(bf16_lo(a.x), bf16_lo(a.y)), f2(bf16_lo(b.x), bf16_lo(b.y))},
                {f2(bf16_hi(a.x), bf16_hi(a.y)), f2(bf16_hi(b.x), bf16_hi(b.y))}};
    else
        return {{f2(bf16_lo(a.x), bf16_hi(a.x)), f2(bf16_lo(a.y), bf16_hi(a.y))},
                {f2(bf16_lo(b.x), bf16_hi(b.x)), f2(bf16_lo(b.y), bf16_hi(b.y))}};
}
template <bool PAIRS>
__device__ __forceinline__ QkPairs qk_get(const QkRaw<float> &r) {
    const float4 a = r.c[0], b = r.c[1];
    if constexpr (PAIRS)
        return {{f2(a.x, a.z), f2(b.x, b.z)}, {f2(a.y, a.w), f2(b.y, b.w)}};
    else
        return {{f2(a.x, a.y), f2(a.z, a.w)}, {f2(b.x, b.y), f2(b.z, b.w)}};
}
template <class T, bool PAIRS>
__device__ __forceinline__ QkRaw<T> qk_put(const QkPairs &p) {
    const float2 x0 = f2_get(p.x[0]), x1 = f2_get(p.x[1]), y0 = f2_get(p.y[0]), y1 = f2_get(p.y[1]);
    if constexpr (sizeof(T) == 4) {
        if constexpr (PAIRS)
            return {{make_float4(x0.x, y0.x, x0.y, y0.y), make_float4(x1.x, y1.x, x1.y, y1.y)}};
        else
            return {{make_float4(x0.x, x0.y, x1.x, x1.y), make_float4(y0.x, y0.y, y1.x, y1.y)}};
    } else {
        if constexpr (PAIRS)
            return {{make_uint2(bf16_pair(x0.x, y0.x), bf16_pair(x0.y, y0.y)), make_uint2(bf16_pair(x1.x, y1.x), bf16_pair(x1.y, y1.y))}};
        else
            return {{make_uint2(bf16_pair(x0.x, x0.y), bf16_pair(x1.x, x1.y)), make_uint2(bf16_pair(y0.x, y0.y), bf16_pair(y1.x, y1.y))}};
    }
}

// Where slot s's two chunks are in a head, and whether they are rotated (by angles `angle` ... + 3).  A lane
// without a slot reads what the first one does.
struct QkSlot {
    int c0, c1, angle;
    bool live, turned;
};
template <bool PAIRS>
__device__ __forceinline__ QkSlot qk_slot(const QkArgs &a, int s) {
    QkSlot q;
    q.live = s < a.D / 8;
    if (!q.live) s = 0;
    q.turned = s < a.R / 8;
    q.angle = 4 * s;
    if (PAIRS) {
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
// Where element e (0..7: x[0], x[1], y[0], y[1] of QkPairs) of a slot is in its head.
template <bool PAIRS>
__device__ __forceinline__ int qk_place(const QkSlot &q, int e) {
    if (PAIRS) return q.c0 + 2 * (e & 3) + (e >> 2);
    return e < 4 ? q.c0 + e : q.c1 + e - 4;
}

template <class T>
__device__ __forceinline__ QkRaw<T> qk_load(const void *base, int64_t at, const QkSlot &q) {
    using Chunk = std::remove_reference_t<decltype(QkRaw<T>{}.c[0])>;
    const T *p = static_cast<const T *>(base) + at;
    QkRaw<T> r;
    r.c[0] = *reinterpret_cast<const Chunk *>(p + q.c0);
    r.c[1] = *reinterpret_cast<const Chunk *>(p + q.c1);
    return r;
}
template <class T>
__device__ __forceinline__ void qk_store(const QkArgs &a, int64_t at, const QkSlot &q, const QkRaw<T> &r) {
    using Chunk = std::remove_reference_t<decltype(QkRaw<T>{}.c[0])>;
    T *const base = static_cast<T *>(a.y);
    const int64_t size = ((a.T - 1) * a.ldy + (int64_t)(a.heads[0] + a.heads[1] - 1) * a.hsy + a.D) * (int64_t)sizeof(T);
    T *const p = base + at;
    if (QT2_STORE_OK(p + q.c0, 4 * sizeof(T), base, size)) *reinterpret_cast<Chunk *>(p + q.c0) = r.c[0];
    if (QT2_STORE_OK(p + q.c1, 4 * sizeof(T), base, size)) *reinterpret_cast<Chunk *>(p + q.c1) = r.c[1];
}
template <bool PAIRS>
__device__ __forceinline__ QkPairs qk_weight(const QkArgs &a, int kind, const QkSlot &q) {
    const void *p = a.w[kind];
    const uint64_t one = f2(1.0f, 1.0f);
    if (!p || !q.live) return {{one, one}, {one, one}};
    return a.w_f32 ? qk_get<PAIRS>(qk_load<float>(p, 0, q)) : qk_get<PAIRS>(qk_load<__nv_bfloat16>(p, 0, q));
}
// cos and sin of four pairs; 1 and 0 where nothing is turned.
struct QkAngles {
    uint64_t c[2], s[2];
};
__device__ __forceinline__ QkAngles qk_angles(const QkArgs &a, int64_t pos, const QkSlot &q) {
    float4 c = make_float4(1.0f, 1.0f, 1.0f, 1.0f), d = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (q.turned && (uint64_t)pos < (uint64_t)a.P) {
        const int64_t at = pos * (a.R / 2) + q.angle;
        c = *reinterpret_cast<const float4 *>(a.cos + at);
        d = *reinterpret_cast<const float4 *>(a.sin + at);
    }
    return {{f2(c.x, c.y), f2(c.z, c.w)}, {f2(d.x, d.y), f2(d.z, d.w)}};
}
// (x, y) -> (x c - y s, y c + x s), or back.
template <bool BACK>
__device__ __forceinline__ void qk_turn(QkPairs &p, const QkAngles &g) {
    const uint64_t minus = f2(-1.0f, -1.0f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t s = f2_mul(g.s[i], minus), x = p.x[i], y = p.y[i];
        p.x[i] = f2_fma(y, BACK ? g.s[i] : s, f2_mul(x, g.c[i]));
        p.y[i] = f2_fma(x, BACK ? s : g.s[i], f2_mul(y, g.c[i]));
    }
}
__device__ __forceinline__ uint64_t qk_squares(const QkPairs &v, uint64_t sum) {
    return f2_fma(v.x[0], v.x[0], f2_fma(v.x[1], v.x[1], f2_fma(v.y[0], v.y[0], f2_fma(v.y[1], v.y[1], sum))));
}

// What a group of lanes takes at a time: U heads of one kind of one token, which share its angles; the last of
// them again where the kind's heads have no more.
template <int U>
struct QkUnit {
    uint32_t t, h, more;   // token, first head (of all), heads behind it
    __device__ __forceinline__ bool live(int u) const { return (uint32_t)u <= more; }
    __device__ __forceinline__ int64_t at(int u, uint32_t ld, uint32_t hs) const {
        return (int64_t)((uint64_t)t * ld + (uint64_t)h * hs + (uint64_t)min((uint32_t)u, more) * hs);
    }
};
template <int U>
__device__ __forceinline__ uint32_t qk_units(const QkArgs &a, int kind) {   // a token's
    return ((uint32_t)a.heads[kind] + U - 1) / U;
}
template <int U>
__device__ __forceinline__ QkUnit<U> qk_unit(const QkArgs &a, int kind, uint32_t units, uint32_t unit) {
    QkUnit<U> q;
    q.t = unit / units;
    const uint32_t h = (unit - q.t * units) * U;
    q.h = h + (kind ? a.heads[0] : 0);
    q.more = min((uint32_t)U, (uint32_t)a.heads[kind] - h) - 1;
    return q;
}

// Blocks an SM, 32768 x 16+16 x 128 bf16 and 16384 tokens of fp32: 3 and 4 (64 registers) 107 and 97 us, 5 (48, of
// which 12 to 24 bytes are spilled) 105 and 91, 6 (40, 44 to 112 bytes) 120 and 102.
template <class T, int G, int N, int U, bool PAIRS>
__global__ void __launch_bounds__(kQkThreads, N > 1 ? 2 : 5) qk_norm_rope_fwd_kernel(const __grid_constant__ QkArgs a) {
    grid_dependency();
    const int g = threadIdx.x % G;
    const float inv_d = 1.0f / (float)a.D;
    int64_t unit = (int64_t)blockIdx.x * (kQkThreads / G) + threadIdx.x / G;
    // queries' units, filled up to whole warps so that a warp has one kind
    const uint32_t units[2] = {qk_units<U>(a, 0), qk_units<U>(a, 1)};
    const int64_t queries = (a.T * units[0] + 32 / G - 1) / (32 / G) * (32 / G);
    const int kind = unit >= queries;
    if (kind) unit -= queries;
    const int64_t all = a.T * units[kind];
    const bool live = unit < all;
    if (!__any_sync(0xFFFFFFFFu, live)) return;
    const QkUnit<U> q = qk_unit<U>(a, kind, units[kind], live ? (uint32_t)unit : (uint32_t)all - 1);
    const int64_t pos = a.pos ? a.pos[q.t] : q.t;
    QkSlot slot[N];
    QkRaw<T> raw[U][N];
    QkAngles angle[N];
    QkPairs w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i] = qk_slot<PAIRS>(a, g + i * G);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i) raw[u][i] = qk_load<T>(a.x, q.at(u, a.ldx, a.hsx), slot[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = qk_weight<PAIRS>(a, kind, slot[i]);
        angle[i] = qk_angles(a, pos, slot[i]);
    }
    if (a.R && live && (uint64_t)pos >= (uint64_t)a.P) set_device_error(QT2_ERR_INVALID_ARG);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        QkPairs v[N];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = qk_get<PAIRS>(raw[u][i]);
            const float part = f2_sum(qk_squares(v[i], 0));
            sum += slot[i].live ? part : 0.0f;
        }
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float r = rsqrtf(fmaf(sum, inv_d, a.eps));
        const uint64_t r2 = f2(r, r);
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[i].x[e] = f2_mul(f2_mul(v[i].x[e], r2), w[i].x[e]);
                v[i].y[e] = f2_mul(f2_mul(v[i].y[e], r2), w[i].y[e]);
            }
            qk_turn<false>(v[i], angle[i]);
            if (live && slot[i].live && q.live(u))
                qk_store<T>(a, q.at(u, a.ldy, a.hsy), slot[i], qk_put<T, PAIRS>(v[i]));
        }
    }
}

// part[block][kind][D]: the block's share of dw.
template <class T, int G, int N, int U, bool PAIRS>
__global__ void __launch_bounds__(kQkThreads, N > 1 ? 1 : 2) qk_norm_rope_bwd_kernel(const __grid_constant__ QkArgs a) {
    constexpr int kWarps = kQkThreads / 32, kGroups = 32 / G;
    extern __shared__ float sums[];   // [kWarps][D]
    grid_dependency();
    const int lane = threadIdx.x & 31, g = lane % G, warp = threadIdx.x >> 5;
    const float inv_d = 1.0f / (float)a.D;
    QkSlot slot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i] = qk_slot<PAIRS>(a, g + i * G);
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        QkPairs w[N], acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = qk_weight<PAIRS>(a, kind, slot[i]);
            acc[i] = QkPairs{};
        }
        const uint32_t units = qk_units<U>(a, kind);
        const int64_t all = a.T * units;
#pragma unroll 1
        for (int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * kGroups; first < all; first += (int64_t)gridDim.x * kWarps * kGroups) {
            const int64_t unit = first + lane / G;
            const bool live = unit < all;
            const QkUnit<U> q = qk_unit<U>(a, kind, units, live ? (uint32_t)unit : (uint32_t)all - 1);
            const int64_t pos = a.pos ? a.pos[q.t] : q.t;
            QkRaw<T> raw[U][N], up[U][N];
            QkAngles angle[N];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    raw[u][i] = qk_load<T>(a.x, q.at(u, a.ldx, a.hsx), slot[i]);
                    up[u][i] = qk_load<T>(a.dy, q.at(u, a.lddy, a.hsdy), slot[i]);
                }
#pragma unroll
            for (int i = 0; i < N; ++i) angle[i] = qk_angles(a, pos, slot[i]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                QkPairs v[N], b[N];
                float sum = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    v[i] = qk_get<PAIRS>(raw[u][i]);
                    b[i] = qk_get<PAIRS>(up[u][i]);
                    qk_turn<true>(b[i], angle[i]);
                    uint64_t dot2 = 0;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        dot2 = f2_fma(f2_mul(b[i].x[e], w[i].x[e]), v[i].x[e], dot2);
                        dot2 = f2_fma(f2_mul(b[i].y[e], w[i].y[e]), v[i].y[e], dot2);
                    }
                    const float part = f2_sum(qk_squares(v[i], 0)), share = f2_sum(dot2);
                    sum += slot[i].live ? part : 0.0f;
                    dot += slot[i].live ? share : 0.0f;
                }
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) {
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
                }
                const float r = rsqrtf(fmaf(sum, inv_d, a.eps));
                const float minus_mean = -(dot * r * inv_d);   // of b w n
                const uint64_t r2 = f2(r, r), m2 = f2(minus_mean, minus_mean);
                const bool row = live && q.live(u);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    QkPairs d;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint64_t nx = f2_mul(v[i].x[e], r2), ny = f2_mul(v[i].y[e], r2);
                        d.x[e] = f2_mul(r2, f2_fma(nx, m2, f2_mul(b[i].x[e], w[i].x[e])));
                        d.y[e] = f2_mul(r2, f2_fma(ny, m2, f2_mul(b[i].y[e], w[i].y[e])));
                        if (row) {
                            acc[i].x[e] = f2_fma(b[i].x[e], nx, acc[i].x[e]);
                            acc[i].y[e] = f2_fma(b[i].y[e], ny, acc[i].y[e]);
                        }
                    }
                    if (a.y && slot[i].live && row)
                        qk_store<T>(a, q.at(u, a.ldy, a.hsy), slot[i], qk_put<T, PAIRS>(d));
                }
            }
        }
        if (!a.part) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 p[4] = {f2_get(acc[i].x[0]), f2_get(acc[i].x[1]), f2_get(acc[i].y[0]), f2_get(acc[i].y[1])};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = e & 1 ? p[e / 2].y : p[e / 2].x;
#pragma unroll
                for (int o = G; o < 32; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                if (lane < G && slot[i].live) sums[warp * a.D + qk_place<PAIRS>(slot[i], e)] = x;
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
