// norm_kernels.cuh -- layer norm forward and backward.
//
//   mean = sum x / C, rstd = 1/sqrt(sum (x - mean)^2 / C + eps), y = (x - mean) rstd w + b
//   h = (x - mean) rstd, a = dy w:  dx = rstd (a - sum a / C - h sum(a h) / C)
//   dw = sum_r dy h, db = sum_r dy
//
// HBM bounds all of it from some MB on, launches below.  Measured (B200, inputs larger than L2, a copy
// of as many bytes at 6.0-6.3 TB/s; calls back to back, 1 to 6 us more where inputs change from call to call):
// forward 16384 x 4096 bf16 51 us (5.3 TB/s), 32768 x 2048 bf16 46 us (5.9), 16384 x 4096 fp32 92 us (5.9);
// backward 32768 x 2048 bf16 64 us for dx (6.3), 70 us with dw and db, 16384 x 4096 fp32 121 and 127 us (6.7),
// 4096 x 16384 bf16 84 and 102 us (4.8).  Rows of more than 16384 columns are read again for each pass: 2048 x
// 20000 bf16 forward 58 us (2.8), backward 58 us for dx (4.2), 128 us with dw and db, which read x and dy from
// HBM once more, a column a thread.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"
#include "vec_device.cuh"

namespace qt2 {

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

constexpr int kNormThreads = 512;   // of the kernels for rows too long for registers

// 16 bytes of a row: 8 bf16 or 4 fp32 elements.
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// Elements [c, c + E) of a weight vector of either type (`other` where there is none).  No 16 bytes
// without an element of the vector are touched.  Plain loads, as everywhere in these kernels: the kernel
// before this one may have written the vector while this one was already resident, and a read-only load
// is not bound by the wait for it.
template <int E>
__device__ __forceinline__ void load_weight(const void *w, int f32, int c, int cols, float other, float (&v)[E]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = other;
    } else if (f32) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c + e);
            const float4 q = c + e < cols ? *p : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            v[e] = q.x; v[e + 1] = q.y; v[e + 2] = q.z; v[e + 3] = q.w;
        }
    } else if constexpr (E == 8) {
        unpack(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(w) + c), v);
    } else {
        const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(w) + c);
        v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    }
    if (c + E > cols) {   // what lies behind the vector may be NaN
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c + e >= cols) v[e] = other;
    }
}

// Writes elements [c, c + E) of a row that are below cols.
template <class T, bool WHOLE = false>
__device__ __forceinline__ void store_row(T *row, int c, int cols, const float (&v)[kVec<T>], const void *base,
                                          int64_t extent) {
    if (c >= cols) return;
    const int n = WHOLE ? kVec<T> : min(kVec<T>, cols - c);
    if (!QT2_STORE_OK(row + c, n * sizeof(T), base, extent * sizeof(T))) return;
    if (n == kVec<T>) {
        *reinterpret_cast<uint4 *>(row + c) = pack(v);
    } else {
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e)
            if (e < n) row[c + e] = from_f32<T>(v[e]);
    }
}

// Pairs of fp32 values in a 64-bit register, and the packed instructions on them: they halve the
// instructions an element costs, which is what bounds these kernels next to HBM.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_get(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float f2_sum(uint64_t v) {
    const float2 p = f2_get(v);
    return p.x + p.y;
}
// The pairs of a 16-byte vector, and back (rounded to the row's type).
__device__ __forceinline__ uint64_t bf16_pair_f2(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }
template <class T>
__device__ __forceinline__ void pairs_of(const uint4 &r, uint64_t (&v)[kVec<T> / 2]) {
    if constexpr (kVec<T> == 8) {
        v[0] = bf16_pair_f2(r.x); v[1] = bf16_pair_f2(r.y); v[2] = bf16_pair_f2(r.z); v[3] = bf16_pair_f2(r.w);
    } else {
        v[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
        v[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
}
template <int E>
__device__ __forceinline__ void floats_of(const uint64_t (&p)[E / 2], float (&v)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float2 q = f2_get(p[e / 2]);
        v[e] = q.x;
        v[e + 1] = q.y;
    }
}

// Sums of N values (a power of two) over the G threads of a row, the same in each of them.  Within
// a warp the values are scattered over the lanes while they are added: each of the first log2 N
// exchanges halves the values a lane still holds.  The warps of a longer row's group of threads (the
// block, or barrier `bar`'s G threads of it) meet at a barrier; the slot alternates between calls, so
// one barrier a call is enough.
template <int G>
__device__ __forceinline__ void group_sync(int bar) {
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(G) : "memory");
}
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (&sh)[2][32][N], int slot, int bar = 0) {
    constexpr int W = G < 32 ? G : 32;
    const int lane = threadIdx.x & 31;
    static_assert(N <= W && (N & (N - 1)) == 0, "values scatter over the lanes");
    int o = W / 2;
#pragma unroll
    for (int n = N / 2; n > 0; n >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
            v[i] = mine + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
    }
    // v[0] is value i's partial sum, i the lane's top log2 N bits within the row's lanes
    float t = v[0];
#pragma unroll
    for (; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if constexpr (G > 32) {
        constexpr int kWarps = G / 32, kEach = 32 / N;   // lanes that hold a value
        if (lane % kEach == 0) sh[slot][(threadIdx.x % G) >> 5][lane / kEach] = t;
        group_sync<G>(bar);
        // kEach lanes a value add up the warps' sums
        t = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w += kEach)
            if (w + lane % kEach < kWarps) t += sh[slot][w + lane % kEach][lane / kEach];
#pragma unroll
        for (int d = kEach / 2; d > 0; d >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = N == 1 ? t : __shfl_sync(0xFFFFFFFFu, t, (lane & ~(W - 1)) + n * (W / N));
}

struct NormArgs {
    const void *x, *dy, *w, *b;
    void *y;             // forward: y; backward: dx
    float *mean, *rstd;
    int64_t rows, ldx, lddy, ldy;
    int cols, w_f32;
    int warps;           // forward: warps of a block that have rows
    int slots;           // forward, groups of threads: rows on their way
    float eps;
    float *part;         // [splits][2][cols]; backward: null where neither dw nor db is wanted
    int splits;
    int cluster;         // backward: the blocks of the launch are one cluster of so many, which needs no part
    void *dw, *db;
};

// Vector c / E of a row, zeros behind the row's end.
template <class T>
__device__ __forceinline__ uint4 load_row(const T *row, int c, int cols, bool live) {
    constexpr int E = kVec<T>;
    if (!live || c >= cols) return make_uint4(0, 0, 0, 0);
    uint4 r = *reinterpret_cast<const uint4 *>(row + c);
    if (c + E > cols) {   // only a row's last vector
        float v[E];
        unpack(r, v);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c + e >= cols) v[e] = 0.0f;
        r = pack(v);
    }
    return r;
}

// Vector i of a row in shared memory, zeros behind the row's end.
template <class T>
__device__ __forceinline__ uint4 stage_vec(const uint4 *stage, int i, int cols) {
    return load_row(reinterpret_cast<const T *>(stage), i * kVec<T>, cols, true);
}

// Keeps the compiler from holding a vector's unpacked values across this point: unpacking again is
// cheaper than the registers (16 vectors of bf16 a lane would take 128).
__device__ __forceinline__ void repack(uint4 &r) { asm volatile("" : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)); }

// ---------------------------------------------------------------------------------------------
// Forward, rows of up to 16 vectors: G lanes of a warp a row, one vector a lane, B rows at a time, the
// lane's weights and biases in registers.  (A warp a row leaves most lanes without work: 1048576 x 64
// bf16 took 282 us.)
// ---------------------------------------------------------------------------------------------
template <class T, int G, int B>
__global__ void __launch_bounds__(256) layernorm_fwd_short_kernel(const NormArgs a) {
    constexpr int E = kVec<T>, P = E / 2, kGroups = 256 / G;
    grid_dependency();
    const int lane = threadIdx.x % G, group = threadIdx.x / G, c = lane * E;
    float none[2][32][B], wf[E], bf[E];
    load_weight(c < a.cols ? a.w : nullptr, a.w_f32, c, a.cols, 1.0f, wf);
    load_weight(c < a.cols ? a.b : nullptr, a.w_f32, c, a.cols, 0.0f, bf);
    const int64_t stride = (int64_t)gridDim.x * kGroups * B;
    uint4 raw[B];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int k = 0; k < B; ++k)
            raw[k] = load_row(static_cast<const T *>(a.x) + (r0 + k) * a.ldx, c, a.cols, r0 + k < a.rows);
    };
    int64_t at = (int64_t)blockIdx.x * kGroups * B;
    fetch(at + group * B);
    // the trip count is the block's, not the group's: every lane of a warp meets the shuffles of row_sum
    for (; at < a.rows; at += stride) {
        const int64_t r0 = at + group * B;
        uint64_t x[B][P];
        float s[B], mean[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            pairs_of<T>(raw[k], x[k]);
            uint64_t s2 = x[k][0];
#pragma unroll
            for (int e = 1; e < P; ++e) s2 = f2_add(s2, x[k][e]);
            s[k] = f2_sum(s2);
        }
        fetch(r0 + stride);
        row_sum<G>(s, none, 0);
#pragma unroll
        for (int k = 0; k < B; ++k) {
            mean[k] = s[k] / a.cols;
            float q = 0.0f;
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 v = f2_get(x[k][e]);
                const float d0 = c + 2 * e < a.cols ? v.x - mean[k] : 0.0f;
                const float d1 = c + 2 * e + 1 < a.cols ? v.y - mean[k] : 0.0f;
                q = fmaf(d0, d0, fmaf(d1, d1, q));
                x[k][e] = f2(d0, d1);
            }
            s[k] = q;
        }
        row_sum<G>(s, none, 0);
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (r0 + k >= a.rows) continue;
            const float rstd = 1.0f / sqrtf(s[k] / a.cols + a.eps);
            float o[E];
            floats_of<E>(x[k], o);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(o[e] * rstd, wf[e], bf[e]);
            store_row(static_cast<T *>(a.y) + (r0 + k) * a.ldy, c, a.cols, o, a.y, (a.rows - 1) * a.ldy + a.cols);
            if (lane == 0) {
                if (a.mean) put(a.mean, (int64_t)(r0 + k), a.rows, mean[k]);
                if (a.rstd) put(a.rstd, (int64_t)(r0 + k), a.rows, rstd);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Forward, a warp a row (short rows: B of them at a time), V vectors of 16 bytes a lane: one read and
// one write of HBM, no barrier between rows.  A bulk copy brings a warp's next row into its part of
// shared memory while this row, in packed registers, goes through its three passes (mean, squared
// differences, result): without it every warp waits for its row, then computes, and HBM idles meanwhile
// (16384 x 4096 bf16: 58 us).  Weights and biases wait in shared memory as fp32, the vectors' first and
// second halves apart, so that a warp's 16-byte reads touch every bank once; read from global memory
// for each row they cost more L1 wavefronts than the row itself.
// ---------------------------------------------------------------------------------------------
template <class T>
__host__ __device__ inline int norm_row_bytes(int cols) { return (cols * (int)sizeof(T) + 15) / 16 * 16; }

template <class T, int V, int B>
__global__ void __launch_bounds__(256, V *B < 16 ? 3 : 2) layernorm_fwd_kernel(const NormArgs a) {
    constexpr int E = kVec<T>, P = E / 2, Q = E / 4;
    extern __shared__ float4 weights[];   // [2 (weight, bias)][Q][32 V], then B rows a warp
    __shared__ __align__(8) uint64_t full[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = a.warps;
    int64_t row = ((int64_t)blockIdx.x * warps + warp) * B;
    const int64_t stride = (int64_t)gridDim.x * warps * B;
    const uint4 *stage = reinterpret_cast<const uint4 *>(weights + 2 * Q * 32 * V) + warp * B * 32 * V;
    const uint32_t bar = smem_u32(full + warp);
    const int row_bytes = norm_row_bytes<T>(a.cols);
    auto issue = [&](int64_t r) {
        if (r >= a.rows) return;
        const int n = (int)min((int64_t)B, a.rows - r);
        mbar_arrive_expect_tx(bar, n * row_bytes);
        for (int k = 0; k < n; ++k)
            bulk_load(smem_u32(stage + k * 32 * V), static_cast<const T *>(a.x) + (r + k) * a.ldx, row_bytes, bar);
    };
    if (lane == 0 && warp < warps) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    grid_dependency();
    if (lane == 0 && warp < warps) issue(row);
#pragma unroll
    for (int j = 0; j < (V + 7) / 8; ++j) {   // by all of the block's threads: 256
        const int i = (int)threadIdx.x + j * 256;
        if (i >= 32 * V || i * E >= a.cols) continue;
        float w[E], b[E];
        load_weight(a.w, a.w_f32, i * E, a.cols, 1.0f, w);
        load_weight(a.b, a.w_f32, i * E, a.cols, 0.0f, b);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            weights[q * 32 * V + i] = make_float4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            weights[(Q + q) * 32 * V + i] = make_float4(b[4 * q], b[4 * q + 1], b[4 * q + 2], b[4 * q + 3]);
        }
    }
    __syncthreads();
    if (warp >= warps) return;
    float none[2][32][B];
    uint32_t phase = 0;
    bool ok = true;   // after a wait that ran out (reported), the rest is not waited for
    for (; row < a.rows; row += stride) {
        if (ok) ok = mbar_wait_warp(bar, phase);
        phase ^= 1;
        uint4 raw[B][V];
#pragma unroll
        for (int k = 0; k < B; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                raw[k][i] = load_row(reinterpret_cast<const T *>(stage + k * 32 * V), (lane + i * 32) * E, a.cols,
                                     row + k < a.rows);
        __syncwarp();
        if (lane == 0 && ok) issue(row + stride);   // (none follows a wait that ran out)
        float s[B], mean[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            uint64_t s2[2] = {};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                uint64_t v[P];
                pairs_of<T>(raw[k][i], v);
#pragma unroll
                for (int e = 0; e < P; ++e) s2[e & 1] = f2_add(s2[e & 1], v[e]);
            }
            s[k] = f2_sum(f2_add(s2[0], s2[1]));
        }
        row_sum<32>(s, none, 0);
#pragma unroll
        for (int k = 0; k < B; ++k) {
            mean[k] = s[k] / a.cols;
            const uint64_t neg = f2(-mean[k], -mean[k]);
            uint64_t s2[2] = {};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (lane + i * 32) * E;
                uint64_t v[P];
                repack(raw[k][i]);
                pairs_of<T>(raw[k][i], v);
                if (c + E <= a.cols) {
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const uint64_t d = f2_add(v[e], neg);
                        s2[e & 1] = f2_fma(d, d, s2[e & 1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const float2 x = f2_get(v[e]);
                        const uint64_t d = f2(c + 2 * e < a.cols ? x.x - mean[k] : 0.0f,
                                              c + 2 * e + 1 < a.cols ? x.y - mean[k] : 0.0f);
                        s2[e & 1] = f2_fma(d, d, s2[e & 1]);
                    }
                }
            }
            s[k] = f2_sum(f2_add(s2[0], s2[1]));
        }
        row_sum<32>(s, none, 0);
#pragma unroll
        for (int k = 0; k < B; ++k) s[k] = 1.0f / sqrtf(s[k] / a.cols + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (lane + i * 32) * E;
            if (c >= a.cols) continue;
            uint64_t w[P], b[P];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const float4 p = weights[q * 32 * V + lane + i * 32], r = weights[(Q + q) * 32 * V + lane + i * 32];
                w[2 * q] = f2(p.x, p.y);
                w[2 * q + 1] = f2(p.z, p.w);
                b[2 * q] = f2(r.x, r.y);
                b[2 * q + 1] = f2(r.z, r.w);
            }
#pragma unroll
            for (int k = 0; k < B; ++k) {
                if (row + k >= a.rows) continue;
                const uint64_t neg = f2(-mean[k], -mean[k]), r2 = f2(s[k], s[k]);
                uint64_t v[P];
                repack(raw[k][i]);
                pairs_of<T>(raw[k][i], v);
#pragma unroll
                for (int e = 0; e < P; ++e) v[e] = f2_fma(f2_mul(f2_add(v[e], neg), r2), w[e], b[e]);
                float o[E];
                floats_of<E>(v, o);
                store_row(static_cast<T *>(a.y) + (row + k) * a.ldy, c, a.cols, o, a.y,
                          (a.rows - 1) * a.ldy + a.cols);
            }
        }
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < B; ++k) {
                if (row + k >= a.rows) continue;
                if (a.mean) put(a.mean, (int64_t)(row + k), a.rows, mean[k]);
                if (a.rstd) put(a.rstd, (int64_t)(row + k), a.rows, s[k]);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Forward, longer rows: a group of G threads a row, V vectors a thread, one block of 1024 threads an SM.
// Bulk copies bring the next rows into the group's `slots` in shared memory while this one, in
// registers, is worked on.  Weights and biases: in registers where a thread has 16 columns (HOLD), else
// in shared memory, once a block, as in layernorm_fwd_kernel.
// ---------------------------------------------------------------------------------------------
template <class T, int G, int V, bool HOLD>
__global__ void __launch_bounds__(1024, 1) layernorm_fwd_group_kernel(const NormArgs a) {
    constexpr int E = kVec<T>, P = E / 2, Q = E / 4, kGroups = 1024 / G, kMost = 3;
    extern __shared__ float4 weights[];   // !HOLD: [2 (weight, bias)][Q][G V]; then [groups][slots][row]
    __shared__ float sh_all[kGroups][2][32][1];
    __shared__ __align__(8) uint64_t full_all[kGroups][kMost];
    const int cols = a.cols, row_bytes = norm_row_bytes<T>(cols), slots = a.slots;
    const int group = threadIdx.x / G, lane = threadIdx.x % G, bar = group + 1;
    const uint8_t *const ring =
        reinterpret_cast<const uint8_t *>(weights + (HOLD ? 0 : 2 * Q * G * V)) + (size_t)group * slots * row_bytes;
    const uint32_t full0 = smem_u32(full_all[group]);
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int64_t row = (int64_t)blockIdx.x * kGroups + group;
    auto issue = [&](int64_t r, int st) {
        if (r >= a.rows) return;
        mbar_arrive_expect_tx(full0 + 8 * st, row_bytes);
        bulk_load(smem_u32(ring + st * row_bytes), static_cast<const T *>(a.x) + r * a.ldx, row_bytes, full0 + 8 * st);
    };
    if (lane == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(full0 + 8 * i, 1);
        fence_mbar_init();
    }
    grid_dependency();
    if (lane == 0)
        for (int i = 0; i < slots; ++i) issue(row + i * step, i);
    uint64_t w[HOLD ? V : 1][P], b[HOLD ? V : 1][P];
    auto pairs = [&](const float (&f)[E], uint64_t (&p)[P]) {
#pragma unroll
        for (int e = 0; e < P; ++e) p[e] = f2(f[2 * e], f[2 * e + 1]);
    };
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (lane + i * G) * E;
            float f[E];
            load_weight(c < cols ? a.w : nullptr, a.w_f32, c, cols, 1.0f, f);
            pairs(f, w[i]);
            load_weight(c < cols ? a.b : nullptr, a.w_f32, c, cols, 0.0f, f);
            pairs(f, b[i]);
        }
    } else {
        for (int i = threadIdx.x; i < G * V && i * E < cols; i += 1024) {
            float f[E], g[E];
            load_weight(a.w, a.w_f32, i * E, cols, 1.0f, f);
            load_weight(a.b, a.w_f32, i * E, cols, 0.0f, g);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                weights[q * G * V + i] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
                weights[(Q + q) * G * V + i] = make_float4(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]);
            }
        }
    }
    __syncthreads();
    int st = 0, phase = 0, left = 0;
    bool ok = true;   // after a wait that ran out (reported), the rest is not waited for
    for (; row < a.rows; row += step) {
        if (ok) {
            ok = mbar_wait(full0 + 8 * st, (uint32_t)phase);
            left = ok ? 0 : slots - 1;
        }
        const uint4 *const stage = reinterpret_cast<const uint4 *>(ring + st * row_bytes);
        uint4 raw[V];
        uint64_t s2 = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            raw[i] = stage_vec<T>(stage, lane + i * G, cols);
            uint64_t v[P];
            pairs_of<T>(raw[i], v);
#pragma unroll
            for (int e = 0; e < P; ++e) s2 = f2_add(s2, v[e]);
        }
        float s[1] = {f2_sum(s2)};
        row_sum<G>(s, sh_all[group], 0, bar);
        // every thread has the row in registers: its slot takes the one `slots` on
        if (lane == 0 && ok) issue(row + slots * step, st);
        if (++st == slots) {
            st = 0;
            phase ^= 1;
        }
        // after a wait that ran out: the copies that were on their way behind it, before the block ends
        if (left > 0 && lane == 0 && row + step < a.rows) mbar_wait(full0 + 8 * st, (uint32_t)phase);
        if (left > 0) --left;
        const float mean = s[0] / cols;
        const uint64_t neg = f2(-mean, -mean);
        s2 = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (lane + i * G) * E;
            uint64_t v[P];
            repack(raw[i]);
            pairs_of<T>(raw[i], v);
            if (c + E <= cols) {
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const uint64_t d = f2_add(v[e], neg);
                    s2 = f2_fma(d, d, s2);
                }
            } else {
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const float2 x = f2_get(v[e]);
                    const uint64_t d = f2(c + 2 * e < cols ? x.x - mean : 0.0f,
                                          c + 2 * e + 1 < cols ? x.y - mean : 0.0f);
                    s2 = f2_fma(d, d, s2);
                }
            }
        }
        s[0] = f2_sum(s2);
        row_sum<G>(s, sh_all[group], 1, bar);
        const float rstd = 1.0f / sqrtf(s[0] / cols + a.eps);
        const uint64_t r2 = f2(rstd, rstd);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (lane + i * G) * E;
            if (c >= cols) continue;
            uint64_t v[P];
            repack(raw[i]);
            pairs_of<T>(raw[i], v);
            if constexpr (!HOLD) {
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float4 p = weights[q * G * V + lane + i * G], r = weights[(Q + q) * G * V + lane + i * G];
                    w[0][2 * q] = f2(p.x, p.y);
                    w[0][2 * q + 1] = f2(p.z, p.w);
                    b[0][2 * q] = f2(r.x, r.y);
                    b[0][2 * q + 1] = f2(r.z, r.w);
                }
            }
#pragma unroll
            for (int e = 0; e < P; ++e)
                v[e] = f2_fma(f2_mul(f2_add(v[e], neg), r2), w[HOLD ? i : 0][e], b[HOLD ? i : 0][e]);
            float o[E];
            floats_of<E>(v, o);
            store_row(static_cast<T *>(a.y) + row * a.ldy, c, cols, o, a.y, (a.rows - 1) * a.ldy + cols);
        }
        if (lane == 0) {
            if (a.mean) put(a.mean, (int64_t)(row), a.rows, mean);
            if (a.rstd) put(a.rstd, (int64_t)(row), a.rows, rstd);
        }
    }
}

// Column c of dw, or of db, where it is wanted.
__device__ __forceinline__ void norm_put_weight(const NormArgs &a, bool bias, int c, float v) {
    void *out = bias ? a.db : a.dw;
    if (!out) return;
    if (a.w_f32)
        put(static_cast<float *>(out), (int64_t)c, (int64_t)a.cols, v);
    else
        put(static_cast<__nv_bfloat16 *>(out), (int64_t)c, (int64_t)a.cols, __float2bfloat16_rn(v));
}

// ---------------------------------------------------------------------------------------------
// Backward, rows of up to 64 columns, one read of x and dy and one write of dx: G threads of a warp a
// row, V vectors a thread, B rows at a time; the next rows are on their way while these are reduced and
// written.  A thread keeps its columns (and their weights) for all of the block's rows and sums their
// dw and db in registers; a block leaves one partial sum a column, which layernorm_dw_kernel adds up.
// With d = x - mean the row's sums are sum(a) and sum(a d), and dx = rstd (a - (rstd^2 sum(a d) / C) d -
// sum(a) / C): sum(a d) times rstd once is of a's size, and no power of rstd stands alone, so that rows of
// any deviation that fp32 has stay within it.
// ---------------------------------------------------------------------------------------------
template <class T, int G, int V, int B>
__global__ void __launch_bounds__(256, 2) layernorm_bwd_kernel(const NormArgs a) {
    grid_dependency();
    constexpr int E = kVec<T>, P = E / 2, kThreads = 256, kGroups = kThreads / G;
    __shared__ float sh[2][32][2 * B];
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    uint64_t w[V][P], dw2[V][P] = {}, db2[V][P] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (lane + i * G) * E;
        float f[E];
        load_weight(c < a.cols ? a.w : nullptr, a.w_f32, c, a.cols, 1.0f, f);
#pragma unroll
        for (int e = 0; e < P; ++e) w[i][e] = f2(f[2 * e], f[2 * e + 1]);
    }
    const float inv = 1.0f / a.cols;
    int slot = 0;
    uint4 rx[B][V], rd[B][V];
    float mean[B], rstd[B];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const bool live = r0 + k < a.rows;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (lane + i * G) * E;
                rx[k][i] = load_row(static_cast<const T *>(a.x) + (r0 + k) * a.ldx, c, a.cols, live);
                rd[k][i] = load_row(static_cast<const T *>(a.dy) + (r0 + k) * a.lddy, c, a.cols, live);
            }
            mean[k] = live ? a.mean[r0 + k] : 0.0f;
            rstd[k] = live ? a.rstd[r0 + k] : 0.0f;
        }
    };
    int64_t at = (int64_t)blockIdx.x * kGroups * B;
    const int64_t stride = (int64_t)gridDim.x * kGroups * B;
    fetch(at + group * B);
    // the trip count is the block's, not the group's: every lane of a warp meets the shuffles of row_sum
    for (; at < a.rows; at += stride) {
        const int64_t r0 = at + group * B;
        float s[2 * B], scale[B];
        uint64_t d[B][V][P], p[B][V][P];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const uint64_t neg = f2(-mean[k], -mean[k]), r2 = f2(rstd[k], rstd[k]);
            uint64_t s2 = 0, q2 = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                uint64_t x[P], g[P];
                pairs_of<T>(rx[k][i], x);
                pairs_of<T>(rd[k][i], g);   // zero behind the row's end
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    d[k][i][e] = f2_add(x[e], neg);
                    p[k][i][e] = f2_mul(g[e], w[i][e]);
                    s2 = f2_add(s2, p[k][i][e]);
                    q2 = f2_fma(p[k][i][e], d[k][i][e], q2);
                    db2[i][e] = f2_add(db2[i][e], g[e]);
                    dw2[i][e] = f2_fma(g[e], f2_mul(d[k][i][e], r2), dw2[i][e]);
                }
            }
            s[2 * k] = f2_sum(s2);
            s[2 * k + 1] = f2_sum(q2);
            scale[k] = rstd[k];
        }
        fetch(r0 + stride);
        if (a.y) {
            row_sum<G>(s, sh, slot);
            slot ^= 1;
#pragma unroll
            for (int k = 0; k < B; ++k) {
                if (r0 + k >= a.rows) continue;
                const float m1 = -s[2 * k] * inv, m2 = -s[2 * k + 1] * inv * scale[k] * scale[k];
                const uint64_t m1p = f2(m1, m1), m2p = f2(m2, m2), r2 = f2(scale[k], scale[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int e = 0; e < P; ++e)
                        p[k][i][e] = f2_mul(f2_add(p[k][i][e], f2_fma(d[k][i][e], m2p, m1p)), r2);
                    float o[E];
                    floats_of<E>(p[k][i], o);
                    store_row(static_cast<T *>(a.y) + (r0 + k) * a.ldy, (lane + i * G) * E, a.cols, o, a.y,
                              (a.rows - 1) * a.ldy + a.cols);
                }
            }
        }
    }
    if (!a.part) return;
    float dw[V][E], db[V][E];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        floats_of<E>(dw2[i], dw[i]);
        floats_of<E>(db2[i], db[i]);
    }
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    // the groups' sums meet in shared memory, in the groups' order
    __shared__ float sum[kGroups][G * V * E];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e)
                sum[group][(lane + i * G) * E + e] = which ? db[i][e] : dw[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < min(a.cols, G * V * E); c += kThreads) {
            float t = 0.0f;
#pragma unroll
            for (int q = 0; q < kGroups; ++q) t += sum[q][c];
            put(a.part, part - a.part + which * a.cols + c, (int64_t)a.splits * 2 * a.cols, t);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// The same for rows of more than 64 columns: one block an SM, whose groups of G threads each take B
// rows at a time, V vectors a thread; bulk copies bring the rows of x and dy into the group's ring of
// S slots in shared memory.  In flight is then what shared memory holds, not what registers are left
// for; a row's vectors are read from shared memory twice instead of being held over the row's
// sums.  The groups' sums of dw and db meet in shared memory, so that an SM leaves one partial
// sum a column (from a block a group, 888 of them at 2048 columns, they cost 19 us of 87).  WHOLE: the
// row's length is a multiple of the vector's, so that no vector has to be cut.
// ---------------------------------------------------------------------------------------------
// The parameters for rows of up to C G columns (C = 8: half the vectors, twice the rows).  bf16: two
// rows share the loop's and the sums' instructions, and a deeper ring is worth more than more threads
// (32768 x 2048: one row at a time 94 us, two 79 us; 640 threads and 2 slots 76 us, 512 and 3 slots less).
// fp32 has half the instructions a byte, and twice the bytes to hold.
// C = 32 columns a thread: the weights are in shared memory, which leaves room for two slots of a bf16 row
// and one of an fp32 row.
template <class T, int G, int C>
struct NormRing {
    static constexpr bool k16 = sizeof(T) == 2;
    static constexpr int V = C / kVec<T>;                             // vectors a thread
    static constexpr int B = C == 32 ? 1 : (k16 ? 2 : 1) * 16 / C;    // rows at a time
    static constexpr int S = C == 32 ? (k16 ? 2 : 1) : k16 || G == 512 ? 3 : 2;   // slots of B rows
    static constexpr int kGroups = (k16 || G == 512 ? 512 : 768) / G;
    static constexpr int kColumns = C * G;
    static constexpr bool kHold = C < 32;                             // weights in registers
    static constexpr int kWeights = kHold ? 0 : kColumns * 4;         // bytes of them in shared memory
    static constexpr int bytes(int cols) { return kWeights + kGroups * S * B * 2 * norm_row_bytes<T>(cols); }
};

template <class T, int G, int C, bool WHOLE>
__global__ void __launch_bounds__(NormRing<T, G, C>::kGroups *G, 1) layernorm_bwd_ring_kernel(const NormArgs a) {
    using R = NormRing<T, G, C>;
    constexpr int E = kVec<T>, P = E / 2, Q = E / 4, V = R::V, S = R::S, B = R::B, kGroups = R::kGroups;
    extern __shared__ float4 weights[];   // !kHold: [Q][G V]; then the rings: [groups][S][B][2 (x, dy)][row]
    uint8_t *const ring_all = reinterpret_cast<uint8_t *>(weights) + R::kWeights;
    __shared__ float sh_all[kGroups][2][32][2 * B];
    __shared__ __align__(8) uint64_t full_all[kGroups][S];
    const int cols = a.cols, rows = (int)a.rows, row_bytes = norm_row_bytes<T>(cols);
    const int group = threadIdx.x / G, lane = threadIdx.x % G, bar = group + 1;
    uint8_t *const ring = ring_all + (size_t)group * S * B * 2 * row_bytes;
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(full_all[group]);
    const int step = (int)gridDim.x * kGroups * B;
    // the group's first thread brings rows [r, r + B) into slot st
    auto issue = [&](int r, int st) {
        const int n = min(B, rows - r);
        if (n <= 0) return;
        mbar_arrive_expect_tx(full0 + 8 * st, n * 2 * row_bytes);
        for (int k = 0; k < n; ++k) {
            const uint32_t dst = ring0 + (st * B + k) * 2 * row_bytes;
            bulk_load(dst, static_cast<const T *>(a.x) + (r + k) * a.ldx, row_bytes, full0 + 8 * st);
            bulk_load(dst + row_bytes, static_cast<const T *>(a.dy) + (r + k) * a.lddy, row_bytes, full0 + 8 * st);
        }
    };
    const int first = ((int)blockIdx.x * kGroups + group) * B;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(full0 + 8 * i, 1);
        fence_mbar_init();
    }
    grid_dependency();
    if (lane == 0)
        for (int i = 0; i < (S > 1 ? S - 1 : 1); ++i) issue(first + i * step, i);
    uint64_t held[R::kHold ? V : 1][P], dw2[V][P] = {}, db2[V][P] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (lane + i * G) * E;
        float f[E];
        load_weight(c < cols ? a.w : nullptr, a.w_f32, c, cols, 1.0f, f);
        if constexpr (R::kHold) {
#pragma unroll
            for (int e = 0; e < P; ++e) held[i][e] = f2(f[2 * e], f[2 * e + 1]);
        } else {   // one group: every thread reads back what it wrote
#pragma unroll
            for (int q = 0; q < Q; ++q)
                weights[q * G * V + lane + i * G] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
        }
    }
    auto weight = [&](int v, uint64_t (&w)[P]) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if constexpr (R::kHold) {
                w[2 * q] = held[v][2 * q];
                w[2 * q + 1] = held[v][2 * q + 1];
            } else {
                const float4 p = weights[q * G * V + lane + v * G];
                w[2 * q] = f2(p.x, p.y);
                w[2 * q + 1] = f2(p.z, p.w);
            }
        }
    };
    __syncthreads();
    const float inv = 1.0f / cols;
    bool ok = true;   // after a wait that ran out (reported), the rest is not waited for
    float mean[B], rstd[B], next_mean[B], next_rstd[B];
    auto stats = [&](int r) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            next_mean[k] = r + k < rows ? a.mean[r + k] : 0.0f;
            next_rstd[k] = r + k < rows ? a.rstd[r + k] : 0.0f;
        }
    };
    stats(first);
    int st = 0, phase = 0, slot = 0, left = 0;
    for (int row = first; row < rows; row += step) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            mean[k] = next_mean[k];
            rstd[k] = next_rstd[k];
        }
        stats(row + step);
        if (ok) {
            ok = mbar_wait(full0 + 8 * st, (uint32_t)phase);
            left = ok ? 0 : S - 2;
        }
        const uint4 *const px = reinterpret_cast<const uint4 *>(ring + st * B * 2 * row_bytes);
        // pairs of x - mean and of dy of row k's vector v; zeros behind the row's end
        auto read = [&](int k, int v, uint64_t (&d)[P], uint64_t (&g)[P]) {
            const int at = lane + v * G, c = at * E;
            const uint64_t neg = f2(-mean[k], -mean[k]);
            const uint4 *x = px + 2 * k * (row_bytes >> 4) + at, *y = x + (row_bytes >> 4);
            if (WHOLE || c + E <= cols) {
                pairs_of<T>(*x, d);
                pairs_of<T>(*y, g);
#pragma unroll
                for (int e = 0; e < P; ++e) d[e] = f2_add(d[e], neg);
                return;
            }
            float xf[E], yf[E];
            unpack(*x, xf);
            unpack(*y, yf);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const bool one = c + e < cols, both = c + e + 1 < cols;
                d[e / 2] = f2(one ? xf[e] - mean[k] : 0.0f, both ? xf[e + 1] - mean[k] : 0.0f);
                g[e / 2] = f2(one ? yf[e] : 0.0f, both ? yf[e + 1] : 0.0f);
            }
        };
        float s[2 * B] = {};
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (row + k >= rows) continue;
            const uint64_t r2 = f2(rstd[k], rstd[k]);
            uint64_t s2 = 0, q2 = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if ((lane + v * G) * E >= cols) continue;
                uint64_t d[P], g[P], w[P];
                read(k, v, d, g);
                weight(v, w);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const uint64_t p = f2_mul(g[e], w[e]);
                    s2 = f2_add(s2, p);
                    q2 = f2_fma(p, d[e], q2);
                    db2[v][e] = f2_add(db2[v][e], g[e]);
                    dw2[v][e] = f2_fma(g[e], f2_mul(d[e], r2), dw2[v][e]);
                }
            }
            s[2 * k] = f2_sum(s2);
            s[2 * k + 1] = f2_sum(q2);
        }
        row_sum<G>(s, sh_all[group], slot, bar);
        slot ^= 1;
        if (G == 32) __syncwarp();
        // every thread is past the rows before these: their slot takes the rows S - 1 steps ahead
        if (S > 1 && lane == 0 && ok) issue(row + (S - 1) * step, st == 0 ? S - 1 : st - 1);
        if (a.y) {
#pragma unroll
            for (int k = 0; k < B; ++k) {
                if (row + k >= rows) continue;
                const float m1 = -s[2 * k] * inv, m2 = -s[2 * k + 1] * inv * rstd[k] * rstd[k];
                const uint64_t m1p = f2(m1, m1), m2p = f2(m2, m2), r2 = f2(rstd[k], rstd[k]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = (lane + v * G) * E;
                    if (c >= cols) continue;
                    uint64_t d[P], g[P], w[P];
                    read(k, v, d, g);
                    weight(v, w);
#pragma unroll
                    for (int e = 0; e < P; ++e)
                        g[e] = f2_mul(f2_fma(g[e], w[e], f2_fma(d[e], m2p, m1p)), r2);
                    float o[E];
                    floats_of<E>(g, o);
                    store_row<T, WHOLE>(static_cast<T *>(a.y) + (row + k) * a.ldy, c, cols, o, a.y,
                                        (a.rows - 1) * a.ldy + cols);
                }
            }
        }
        if (S == 1) {   // the only slot is free when every thread has written its part of dx
            group_sync<G>(bar);
            if (lane == 0 && ok) issue(row + step, 0);
        }
        if (++st == S) {
            st = 0;
            phase ^= 1;
        }
        // after a wait that ran out: the copies that were on their way behind it, before the block ends
        if (left > 0 && lane == 0 && row + step < rows) mbar_wait(full0 + 8 * st, (uint32_t)phase);
        if (left > 0) --left;
    }
    if (!a.part) return;
    // the rings' rows are all read: every group leaves its sums at the start of its ring
    __syncthreads();
    float *const mine = reinterpret_cast<float *>(ring);   // [2][cols]
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float dw[E], db[E];
        floats_of<E>(dw2[v], dw);
        floats_of<E>(db2[v], db);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (lane + v * G) * E + e;
            if (c >= cols) continue;
            mine[c] = dw[e];
            mine[cols + c] = db[e];
        }
    }
    __syncthreads();
    float *const sums = reinterpret_cast<float *>(ring_all);   // the first group's: becomes the block's
    for (int c = threadIdx.x; c < 2 * cols; c += kGroups * G) {
        float t = 0.0f;
#pragma unroll
        for (int q = 0; q < kGroups; ++q)
            t += reinterpret_cast<const float *>(ring_all + (size_t)q * S * B * 2 * row_bytes)[c];
        if (a.cluster)
            sums[c] = t;
        else
            put(a.part, (int64_t)blockIdx.x * 2 * cols + c, (int64_t)a.splits * 2 * cols, t);
    }
    if (!a.cluster) return;
    // few rows: the launch is one cluster, whose blocks add up their sums a share of the columns each
    cluster_sync_all();
    const int rank = (int)cluster_ctarank();
    for (int c = rank * kGroups * G + (int)threadIdx.x; c < 2 * cols; c += a.cluster * kGroups * G) {
        float t = 0.0f;
        for (int q = 0; q < a.cluster; ++q)
            t += __uint_as_float(ld_shared_cluster_u32(mapa_shared(smem_u32(sums + c), q)));
        norm_put_weight(a, c >= cols, c >= cols ? c - cols : c, t);
    }
    cluster_sync_all();   // no block leaves while another reads its sums
}

// dw (blockIdx.y = 0) or db: the sum of the partial sums, 32 columns a block, 32 slices of the
// partial sums side by side.
__global__ void __launch_bounds__(1024) layernorm_dw_kernel(const NormArgs a) {
    grid_dependency();
    __shared__ float sh[32][33];
    void *out = blockIdx.y ? a.db : a.dw;
    if (!out) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    float t = 0.0f;
    if (c < a.cols) {
        const float *part = a.part + (int64_t)blockIdx.y * a.cols + c;
#pragma unroll 16
        for (int i = slice; i < a.splits; i += 32) t += part[(int64_t)i * 2 * a.cols];
    }
    sh[slice][threadIdx.x & 31] = t;
    __syncthreads();
    t = sh[threadIdx.x & 31][slice];   // column `slice` of the block's 32, one slice a lane
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    const int d = blockIdx.x * 32 + slice;
    if ((threadIdx.x & 31) != 0 || d >= a.cols) return;
    norm_put_weight(a, blockIdx.y, d, t);
}

// ---------------------------------------------------------------------------------------------
// Rows too long for registers and shared memory: a block a row, which it reads again for each pass (from
// L2 after the first).
// ---------------------------------------------------------------------------------------------
template <class T>
__global__ void __launch_bounds__(kNormThreads) layernorm_fwd_long_kernel(const NormArgs a) {
    grid_dependency();
    constexpr int E = kVec<T>;
    __shared__ float sh[2][32][1];
    const T *x = static_cast<const T *>(a.x) + (int64_t)blockIdx.x * a.ldx;
    float s[1] = {0.0f};
#pragma unroll 4
    for (int c = threadIdx.x * E; c < a.cols; c += kNormThreads * E) {
        float v[E], t = 0.0f;
        unpack(load_row(x, c, a.cols, true), v);
#pragma unroll
        for (int e = 0; e < E; ++e) t += v[e];
        s[0] += t;
    }
    row_sum<kNormThreads>(s, sh, 0);
    const float mean = s[0] / a.cols;
    s[0] = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x * E; c < a.cols; c += kNormThreads * E) {
        float v[E], t = 0.0f;
        unpack(load_row(x, c, a.cols, true), v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = c + e < a.cols ? v[e] - mean : 0.0f;
            t = fmaf(d, d, t);
        }
        s[0] += t;
    }
    row_sum<kNormThreads>(s, sh, 1);
    const float rstd = 1.0f / sqrtf(s[0] / a.cols + a.eps);
#pragma unroll 2
    for (int c = threadIdx.x * E; c < a.cols; c += kNormThreads * E) {
        float v[E], w[E], b[E];
        unpack(load_row(x, c, a.cols, true), v);
        load_weight(a.w, a.w_f32, c, a.cols, 1.0f, w);
        load_weight(a.b, a.w_f32, c, a.cols, 0.0f, b);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
        store_row(static_cast<T *>(a.y) + (int64_t)blockIdx.x * a.ldy, c, a.cols, v, a.y,
                  (a.rows - 1) * a.ldy + a.cols);
    }
    if (threadIdx.x == 0) {
        if (a.mean) put(a.mean, (int64_t)(blockIdx.x), a.rows, mean);
        if (a.rstd) put(a.rstd, (int64_t)(blockIdx.x), a.rows, rstd);
    }
}

template <class T>
__global__ void __launch_bounds__(kNormThreads) layernorm_dx_long_kernel(const NormArgs a) {
    grid_dependency();
    constexpr int E = kVec<T>;
    __shared__ float sh[2][32][2];
    const T *x = static_cast<const T *>(a.x) + (int64_t)blockIdx.x * a.ldx;
    const T *dy = static_cast<const T *>(a.dy) + (int64_t)blockIdx.x * a.lddy;
    const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
    float s[2] = {};
#pragma unroll 2
    for (int c = threadIdx.x * E; c < a.cols; c += kNormThreads * E) {
        float v[E], g[E], w[E], t = 0.0f, q = 0.0f;
        unpack(load_row(x, c, a.cols, true), v);
        unpack(load_row(dy, c, a.cols, true), g);   // zero behind the row's end
        load_weight(a.w, a.w_f32, c, a.cols, 1.0f, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float p = g[e] * w[e];
            t += p;
            q = fmaf(p, (v[e] - mean) * rstd, q);
        }
        s[0] += t;
        s[1] += q;
    }
    row_sum<kNormThreads>(s, sh, 0);
    const float m1 = s[0] / a.cols, m2 = s[1] / a.cols;
#pragma unroll 2
    for (int c = threadIdx.x * E; c < a.cols; c += kNormThreads * E) {
        float v[E], g[E], w[E];
        unpack(load_row(x, c, a.cols, true), v);
        unpack(load_row(dy, c, a.cols, true), g);
        load_weight(a.w, a.w_f32, c, a.cols, 1.0f, w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = rstd * (g[e] * w[e] - m1 - (v[e] - mean) * rstd * m2);
        store_row(static_cast<T *>(a.y) + (int64_t)blockIdx.x * a.ldy, c, a.cols, v, a.y,
                  (a.rows - 1) * a.ldy + a.cols);
    }
}

// Partial sums of dw and db over rows split, split + splits, ...: one vector a thread.
template <class T>
__global__ void __launch_bounds__(kNormThreads) layernorm_dw_long_kernel(const NormArgs a) {
    grid_dependency();
    constexpr int E = kVec<T>;
    const int c = (blockIdx.x * kNormThreads + threadIdx.x) * E;
    if (c >= a.cols) return;
    float dw[E] = {}, db[E] = {};
#pragma unroll 4
    for (int64_t r = blockIdx.y; r < a.rows; r += a.splits) {
        float v[E], g[E];
        unpack(load_row(static_cast<const T *>(a.x) + r * a.ldx, c, a.cols, true), v);
        unpack(load_row(static_cast<const T *>(a.dy) + r * a.lddy, c, a.cols, true), g);
        const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            db[e] += g[e];
            dw[e] = fmaf(g[e], (v[e] - mean) * rstd, dw[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (c + e >= a.cols) continue;
        const int64_t at = (int64_t)blockIdx.y * 2 * a.cols + c + e, n = (int64_t)a.splits * 2 * a.cols;
        put(a.part, at, n, dw[e]);
        put(a.part, at + a.cols, n, db[e]);
    }
}

}  // namespace qt2
