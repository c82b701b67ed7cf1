// adamw_kernels.cuh -- one AdamW step of many tensors, with states in fp32 or in 8 bits.
//
//   g' = g min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p - lr wd p - lr c1 m / (sqrt(v) c2 + eps),  c1 = 1 / (1 - b1^t),  c2 = 1 / sqrt(1 - b2^t)
//
// States in 8 bits are E4M3 codes with an fp32 scale for 256 elements, m / scale and sqrt(v) / scale: the
// root spans the range of v in half as many binades and is what the update divides by.  A step moves v by
// (1 - b2), far less than the codes' spacing, so codes are rounded up or down at random, with probabilities
// that keep their mean; rounded to nearest, v would stay where it is.  The draws are Philox words of
// (seed, tensor, step, element): 16 bits for m, 16 for v.  What decides a code is rounded operation by
// operation (no contraction), so that it is the same wherever it is computed.
//
// A stream over HBM: everything is read and written once, and the clipping takes no pass of its own.  A
// warp takes 256 elements, its lanes 4 neighbours twice, and loads all arrays before it uses any.  The
// list travels in the kernel's parameters.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"
#include "vec_device.cuh"

namespace qt2 {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;                              // elements that share a scale; a warp's at a time
constexpr int kAdamChunk = kAdamThreads / 32 * kAdamBlock;   // elements a block takes at a time
constexpr int kAdamSmall = 32, kAdamLarge = 384;             // tensors a launch's parameters hold

// Bits of AdamTable::flags.
enum { kAdamParamF32 = 1, kAdamGradF32 = 2, kAdamE4m3 = 4, kAdamVectors = 8, kAdamHead = 16 };   // head: bits 4 and 5

template <int N>
struct AdamTable {
    void *param[N];
    float *master[N];          // may be null
    const void *grad[N];
    void *m[N], *v[N];
    float *m_scale[N], *v_scale[N];
    int64_t numel[N];
    int32_t first[N + 1];      // chunks before tensor i
    int32_t id[N];             // the tensor's place in the caller's list
    float decay[N];
    uint8_t flags[N];
    int count;
};

struct AdamArgs {
    const float *lr, *norm;    // norm may be null
    const int64_t *step;
    double log_b1, log_b2;
    float b1, b2, one_b1, one_b2, eps, max_norm;
    uint64_t seed;
};

// Four neighbours as they lie in memory: 4 words (fp32), 2 (bf16) or 1 (E4M3).
struct AdamRaw {
    uint32_t w[4];
};
template <int BYTES>
__device__ __forceinline__ void adam_load(AdamRaw &r, const void *base, int64_t at, bool whole, int64_t n) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + at * BYTES;
    if (whole) {
        if constexpr (BYTES == 4) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
        } else if constexpr (BYTES == 2) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            r.w[0] = q.x; r.w[1] = q.y;
        } else {
            r.w[0] = *reinterpret_cast<const uint32_t *>(p);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (at + e < 0 || at + e >= n) continue;
        if constexpr (BYTES == 4)
            r.w[e] = reinterpret_cast<const uint32_t *>(p)[e];
        else if constexpr (BYTES == 2)
            r.w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[e] << (16 * (e & 1));
        else
            r.w[0] |= (uint32_t)p[e] << (8 * e);
    }
}
__device__ __forceinline__ void adam_get_f32(const AdamRaw &r, float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(r.w[e]);
}
__device__ __forceinline__ void adam_get_bf16(const AdamRaw &r, float (&v)[4]) {
    v[0] = bf16_lo(r.w[0]); v[1] = bf16_hi(r.w[0]); v[2] = bf16_lo(r.w[1]); v[3] = bf16_hi(r.w[1]);
}
__device__ __forceinline__ void adam_get_e4m3(const AdamRaw &r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        asm("{\n\t.reg .b32 h;\n\t.reg .f16 a, b;\n\tcvt.rn.f16x2.e4m3x2 h, %2;\n\tmov.b32 {a, b}, h;\n\t"
            "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
            : "h"((uint16_t)(r.w[0] >> (16 * i))));
    }
}
template <int BYTES>
__device__ __forceinline__ void adam_store(void *base, int64_t at, bool whole, int64_t n, const AdamRaw &r) {
    uint8_t *p = static_cast<uint8_t *>(base) + at * BYTES;
    if (whole) {
        if (!QT2_STORE_OK(p, 4 * BYTES, base, n * BYTES)) return;
        if constexpr (BYTES == 4)
            *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        else if constexpr (BYTES == 2)
            *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
        else
            *reinterpret_cast<uint32_t *>(p) = r.w[0];
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (at + e < 0 || at + e >= n || !QT2_STORE_OK(p + e * BYTES, BYTES, base, n * BYTES)) continue;
        if constexpr (BYTES == 4)
            reinterpret_cast<uint32_t *>(p)[e] = r.w[e];
        else if constexpr (BYTES == 2)
            reinterpret_cast<uint16_t *>(p)[e] = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
        else
            p[e] = (uint8_t)(r.w[0] >> (8 * e));
    }
}
__device__ __forceinline__ void adam_put_f32(void *base, int64_t at, bool whole, int64_t n, const float (&v)[4]) {
    AdamRaw r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r.w[e] = __float_as_uint(v[e]);
    adam_store<4>(base, at, whole, n, r);
}
__device__ __forceinline__ void adam_put_bf16(void *base, int64_t at, bool whole, int64_t n, const float (&v)[4]) {
    AdamRaw r;
    r.w[0] = bf16_pair(v[0], v[1]);
    r.w[1] = bf16_pair(v[2], v[3]);
    adam_store<2>(base, at, whole, n, r);
}

// What the 256 elements of a warp are divided by to reach E4M3's largest number, and that scale.  Elements
// below 2^-100 are zero with their whole block; one of inf or NaN makes the block's scale NaN.
__device__ __forceinline__ void adam_scale(uint32_t top, float &inv, float &scale) {
    const float t = __uint_as_float(top);
    if (top >= 0x7F800000u) {
        inv = 0.0f;
        scale = __uint_as_float(0x7FFFFFFFu);
    } else if (t < kTiny) {
        inv = scale = 0.0f;
    } else {
        inv = __fdiv_rn(448.0f, t);
        scale = __fdiv_rn(t, 448.0f);
    }
}
// |x| * inv, rounded to E4M3 up or down by a 16-bit draw: the fp32 encoding keeps 3 bits of its mantissa, and
// adding the draw to the 20 behind them carries with the right probability.  Below the normal numbers the
// spacing is that of the smallest normal, which is added meanwhile.  Returns an fp32 number that E4M3 holds.
__device__ __forceinline__ float adam_round(float x, float inv, uint32_t draw) {
    const float a = __fmul_rn(fabsf(x), inv);
    const float lift = a < 0x1p-6f ? 0x1p-6f : 0.0f;
    const uint32_t bits = (__float_as_uint(__fadd_rn(a, lift)) + (draw << 4)) & ~0xFFFFFu;
    return copysignf(fminf(__fsub_rn(__uint_as_float(bits), lift), 448.0f), x);
}
__device__ __forceinline__ uint32_t adam_codes(const float (&v)[4]) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
    return lo | (uint32_t)hi << 16;
}

template <int N>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable<N> t,
                                                             const __grid_constant__ AdamArgs a) {
    grid_dependency();
    __shared__ float corr[2];
    const float lr = *a.lr;
    const int64_t step = *a.step;
    float clip = 1.0f;
    if (a.norm) {
        const float n = *a.norm, q = a.max_norm / (n + 1e-6f);
        if (!(fabsf(n) < INFINITY)) return;   // all of the grid: nothing is changed
        clip = q > 1.0f ? 1.0f : q;
    }
    if (step < 1) {
        set_device_error(QT2_ERR_INVALID_ARG);
        return;
    }
    if (threadIdx.x < 2) {   // 1 - b^t = -(exp(t log b) - 1)
        const double left = -expm1((double)step * (threadIdx.x ? a.log_b2 : a.log_b1));
        corr[threadIdx.x] = (float)(threadIdx.x ? sqrt(1.0 / left) : 1.0 / left);
    }
    __syncthreads();
    const float rate = lr * corr[0], c2 = corr[1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int chunk = blockIdx.x; chunk < t.first[t.count]; chunk += gridDim.x) {
        int k = 0, last = t.count - 1;
        while (k < last) {
            const int mid = (k + last + 1) >> 1;
            if (t.first[mid] <= chunk)
                k = mid;
            else
                last = mid - 1;
        }
        const uint32_t flags = t.flags[k];
        const int64_t n = t.numel[k];
        const bool e4m3 = flags & kAdamE4m3;
        // the first element, and (aligned as the vectors are) up to three before the tensor's first
        const int64_t first = (int64_t)(chunk - t.first[k]) * kAdamChunk + warp * kAdamBlock - (flags / kAdamHead);
        if (first >= n) continue;
        const bool p_f32 = flags & kAdamParamF32, g_f32 = flags & kAdamGradF32;
        const float *const master = t.master[k];
        int64_t at[2];
        bool whole[2];
        AdamRaw rg[2] = {}, rp[2] = {}, rm[2] = {}, rv[2] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            at[i] = first + 128 * i + 4 * lane;
            whole[i] = (flags & kAdamVectors) && at[i] >= 0 && at[i] + 4 <= n;
            if (g_f32)
                adam_load<4>(rg[i], t.grad[k], at[i], whole[i], n);
            else
                adam_load<2>(rg[i], t.grad[k], at[i], whole[i], n);
            if (e4m3) {
                adam_load<1>(rm[i], t.m[k], at[i], whole[i], n);
                adam_load<1>(rv[i], t.v[k], at[i], whole[i], n);
            } else {
                adam_load<4>(rm[i], t.m[k], at[i], whole[i], n);
                adam_load<4>(rv[i], t.v[k], at[i], whole[i], n);
            }
            if (master)
                adam_load<4>(rp[i], master, at[i], whole[i], n);
            else if (p_f32)
                adam_load<4>(rp[i], t.param[k], at[i], whole[i], n);
            else
                adam_load<2>(rp[i], t.param[k], at[i], whole[i], n);
        }
        const int64_t block = first / kAdamBlock, blocks = (n + kAdamBlock - 1) / kAdamBlock;
        const float sm = e4m3 ? t.m_scale[k][block] : 0.0f, sv = e4m3 ? t.v_scale[k][block] : 0.0f;
        const float decay = lr * t.decay[k];
        float m[2][4], root[2][4];
        uint32_t top_m = 0, top_v = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float g[4], v[4], p[4];
            if (g_f32)
                adam_get_f32(rg[i], g);
            else
                adam_get_bf16(rg[i], g);
            if (e4m3) {
                adam_get_e4m3(rm[i], m[i]);
                adam_get_e4m3(rv[i], v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    m[i][e] = __fmul_rn(m[i][e], sm);
                    v[e] = __fmul_rn(v[e], sv);
                    v[e] = __fmul_rn(v[e], v[e]);
                }
            } else {
                adam_get_f32(rm[i], m[i]);
                adam_get_f32(rv[i], v);
            }
            if (master || p_f32)
                adam_get_f32(rp[i], p);
            else
                adam_get_bf16(rp[i], p);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float h = __fmul_rn(g[e], clip);
                m[i][e] = __fadd_rn(__fmul_rn(m[i][e], a.b1), __fmul_rn(h, a.one_b1));
                v[e] = __fadd_rn(__fmul_rn(v[e], a.b2), __fmul_rn(__fmul_rn(h, h), a.one_b2));
                root[i][e] = __fsqrt_rn(v[e]);
                p[e] = fmaf(-decay, p[e], p[e]) - __fdividef(rate * m[i][e], fmaf(root[i][e], c2, a.eps));
                top_m = max(top_m, __float_as_uint(m[i][e]) & 0x7FFFFFFFu);
                top_v = max(top_v, __float_as_uint(root[i][e]) & 0x7FFFFFFFu);
            }
            if (master) adam_put_f32(t.master[k], at[i], whole[i], n, p);
            if (p_f32)
                adam_put_f32(t.param[k], at[i], whole[i], n, p);
            else
                adam_put_bf16(t.param[k], at[i], whole[i], n, p);
            if (!e4m3) {
                adam_put_f32(t.m[k], at[i], whole[i], n, m[i]);
                adam_put_f32(t.v[k], at[i], whole[i], n, v);
            }
        }
        if (!e4m3) continue;
        // elements behind the tensor's end are zeros here
        float im, iv, nm, nv;
        adam_scale(__reduce_max_sync(0xFFFFFFFFu, top_m), im, nm);
        adam_scale(__reduce_max_sync(0xFFFFFFFFu, top_v), iv, nv);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t group = (uint64_t)at[i] >> 2;
            const uint4 w4 = philox4x32_10(make_uint4((uint32_t)group, (uint32_t)(group >> 32), (uint32_t)t.id[k], (uint32_t)step),
                                           make_uint2((uint32_t)a.seed, (uint32_t)(a.seed >> 32)));
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            float qm[4], qv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                qm[e] = adam_round(m[i][e], im, w[e] & 0xFFFFu);
                qv[e] = adam_round(root[i][e], iv, w[e] >> 16);
            }
            AdamRaw r;
            r.w[0] = adam_codes(qm);
            adam_store<1>(t.m[k], at[i], whole[i], n, r);
            r.w[0] = adam_codes(qv);
            adam_store<1>(t.v[k], at[i], whole[i], n, r);
        }
        if (lane == 0) {
            put(t.m_scale[k], block, blocks, nm);
            put(t.v_scale[k], block, blocks, nv);
        }
    }
}

}  // namespace qt2
