// adamw_kernels.cuh -- one AdamW step of many tensors, with states in fp32 or in 8 bits.
//
//   g' = g min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p - lr wd p - lr c1 m / (sqrt(v) c2 + eps),  c1 = 1 / (1 - b1^t),  c2 = 1 / sqrt(1 - b2^t)
//
// States in 8 bits are E4M3 codes with an fp32 scale for 256 elements, m / scale and sqrt(v) / scale: the
// root spans the range of v in half as many binades and is what the update divides by.  A step moves v by
// (1 - b2), far less than the codes' spacing, so codes are rounded up or down at random, with probabilities
// that keep their mean (a root's never to zero); rounded to nearest, v would stay where it is.  The draws are Philox words of
// (seed, tensor, step, element): 16 bits for m, 16 for v.  What decides a code is rounded operation by
// operation (no contraction), so that it is the same wherever it is computed.
//
// A stream over HBM: everything is read and written once, and the clipping takes no pass of its own (411M elements:
// fp32 1.81 to 1.87 ms, 6.2 to 6.4 TB/s).  States in 8 bits make it a stream of instructions: 71 an element, of
// them 15 for the draws, issue 70% (with bf16 parameters and gradients and fp32 masters 1.21 to 1.32 ms, 5.0 to 5.5
// TB/s).  A warp takes 256 elements, its lanes 4 neighbours twice, and loads all arrays before it uses any.  The
// list travels in the kernel's parameters; tensors of different types take launches of their own, each
// compiled for its types.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"
#include "vec_device.cuh"

namespace qt2 {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;                              // elements that share a scale; a warp's at a time
constexpr int kAdamChunk = kAdamThreads / 32 * kAdamBlock;   // elements a block takes at a time
constexpr int kAdamSmall = 32, kAdamLarge = 384;             // tensors a launch's parameters hold

// AdamTable::flags: whether the arrays are aligned alike, and how many elements behind a vector they start.
enum { kAdamVectors = 1, kAdamHead = 2 };
// What a tensor's parameter is; with its gradient's type and its states, what a kernel is compiled for.
enum AdamParam { kAdamBf16 = 0, kAdamF32 = 1, kAdamMaster = 2 };

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
    // what both sides of the update's quotient are multiplied by, eps among them: 1, or a power of two that makes a
    // subnormal eps a normal number (adam_rcp takes any other for zero)
    float unit;
    float minus_zero;
    uint32_t key0[10], key1[10];   // Philox's keys of each round
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
// The four as pairs.
__device__ __forceinline__ void adam_get_f32(const AdamRaw &r, uint64_t (&v)[2]) {
    v[0] = f2(__uint_as_float(r.w[0]), __uint_as_float(r.w[1]));
    v[1] = f2(__uint_as_float(r.w[2]), __uint_as_float(r.w[3]));
}
__device__ __forceinline__ void adam_get_bf16(const AdamRaw &r, uint64_t (&v)[2]) {
    v[0] = f2(bf16_lo(r.w[0]), bf16_hi(r.w[0]));
    v[1] = f2(bf16_lo(r.w[1]), bf16_hi(r.w[1]));
}
__device__ __forceinline__ void adam_get_e4m3(const AdamRaw &r, uint64_t (&v)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float x, y;
        asm("{\n\t.reg .b32 h;\n\t.reg .f16 a, b;\n\tcvt.rn.f16x2.e4m3x2 h, %2;\n\tmov.b32 {a, b}, h;\n\t"
            "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(x), "=f"(y)
            : "h"((uint16_t)(r.w[0] >> (16 * i))));
        v[i] = f2(x, y);
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
__device__ __forceinline__ void adam_put_f32(void *base, int64_t at, bool whole, int64_t n, const uint64_t (&v)[2]) {
    const float2 x = f2_get(v[0]), y = f2_get(v[1]);
    adam_store<4>(base, at, whole, n, AdamRaw{{__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y)}});
}
__device__ __forceinline__ void adam_put_bf16(void *base, int64_t at, bool whole, int64_t n, const uint64_t (&v)[2]) {
    const float2 x = f2_get(v[0]), y = f2_get(v[1]);
    adam_store<2>(base, at, whole, n, AdamRaw{{bf16_pair(x.x, x.y), bf16_pair(y.x, y.y), 0, 0}});
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
// a * b, rounded, where the product goes on into a sum: as a fused multiply-add with -0, which changes nothing.  A
// packed product and a packed sum would be contracted into one operation; nz is -0 at run time only, so that
// this one is not taken for a plain product.
__device__ __forceinline__ uint64_t adam_product(uint64_t a, uint64_t b, float nz) { return f2_fma(a, b, f2(nz, nz)); }

__device__ __forceinline__ uint32_t adam_codes(const float (&v)[4]) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
    return lo | (uint32_t)hi << 16;
}
// b * 2^s + c and (b >> (32 - s)) + c as one instruction each.
__device__ __forceinline__ uint32_t adam_up(uint32_t b, uint32_t s, uint32_t c) {
    uint32_t r;
    asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(r) : "r"(b), "r"(1u << s), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t adam_down(uint32_t b, uint32_t s, uint32_t c) {
    uint32_t r;
    asm("mad.hi.u32 %0, %1, %2, %3;" : "=r"(r) : "r"(b), "r"(1u << s), "r"(c));
    return r;
}

// Four elements as E4M3 codes.  Each is x * inv, rounded up or down by a 16-bit draw d from the low (V: high) half
// of its word: the fp32 encoding (sign and magnitude) keeps 3 bits of its mantissa, and adding 2^4 d to the 20
// behind them carries with the right probability; the largest is off 448 by two units at most, which no draw
// carries any further.  Below the normal numbers the spacing is that of the smallest normal, 2^-6, which is
// added meanwhile: a warp without such elements (and zeros count as such) takes the shorter way.
// A root (V) that is not zero keeps the smallest code where it would round to zero: m, drawn by itself, may have
// rounded up to its smallest code there, and a step that divides that by eps or by the next gradient alone is
// hundreds of learning rates (elements 10^5 below their block's largest: 300 within 300 steps; 10^6: 3500; with the
// smallest code 2.4).
template <bool V>
__device__ __forceinline__ float adam_cut(float x, uint32_t word) {
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float((V ? adam_down(word & 0xFFFF0000u, 20, b) : adam_up(word & 0xFFFFu, 4, b)) & ~0xFFFFFu);
}
__device__ __forceinline__ float adam_lift(float x) { return fabsf(x) < 0x1p-6f ? copysignf(0x1p-6f, x) : 0.0f; }
template <bool V>
__device__ __forceinline__ uint32_t adam_round(const float (&x)[4], bool small, const uint4 &w) {
    float y[4];
    if (small) {
        const float l[4] = {adam_lift(x[0]), adam_lift(x[1]), adam_lift(x[2]), adam_lift(x[3])};
        y[0] = __fsub_rn(adam_cut<V>(__fadd_rn(x[0], l[0]), w.x), l[0]);
        y[1] = __fsub_rn(adam_cut<V>(__fadd_rn(x[1], l[1]), w.y), l[1]);
        y[2] = __fsub_rn(adam_cut<V>(__fadd_rn(x[2], l[2]), w.z), l[2]);
        y[3] = __fsub_rn(adam_cut<V>(__fadd_rn(x[3], l[3]), w.w), l[3]);
        if constexpr (V) {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = x[e] > 0.0f ? fmaxf(y[e], 0x1p-9f) : y[e];
        }
    } else {
        y[0] = adam_cut<V>(x[0], w.x);
        y[1] = adam_cut<V>(x[1], w.y);
        y[2] = adam_cut<V>(x[2], w.z);
        y[3] = adam_cut<V>(x[3], w.w);
    }
    return adam_codes(y);
}
// The larger and the smaller magnitude of the three; NaN where one is.
__device__ __forceinline__ float adam_max(float a, float b, float c) {
    float m;
    asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %2;\n\tabs.f32 y, %3;\n\tmax.NaN.f32 %0, %1, x, y;\n\t}" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ float adam_min(float a, float b, float c) {
    float m;
    asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %2;\n\tabs.f32 y, %3;\n\tmin.NaN.f32 %0, %1, x, y;\n\t}" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ float adam_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Of the step, the same for all tensors.
struct AdamStep {
    uint32_t step;
    float lr, rate, c2, clip;
};

// 256 elements of tensor k, from the warp's first one on.  WHOLE: all of them are the tensor's, and its arrays
// aligned alike; else `first` may be up to three before the tensor's first.
template <int N, bool E4M3, AdamParam P, bool GF32, bool WHOLE>
__device__ __forceinline__ void adam_step(const AdamTable<N> &t, int k, int64_t first, const AdamArgs &a,
                                          const AdamStep &j, int lane) {
    constexpr int kState = E4M3 ? 1 : 4, kGrad = GF32 ? 4 : 2;
    const int64_t n = t.numel[k];
    int64_t at[2];
    bool whole[2];
    AdamRaw rg[2], rp[2], rm[2], rv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        at[i] = first + 128 * i + 4 * lane;
        whole[i] = WHOLE || ((t.flags[k] & kAdamVectors) && at[i] >= 0 && at[i] + 4 <= n);
        if constexpr (!WHOLE) rg[i] = rp[i] = rm[i] = rv[i] = AdamRaw{};
        adam_load<kGrad>(rg[i], t.grad[k], at[i], whole[i], n);
        adam_load<kState>(rm[i], t.m[k], at[i], whole[i], n);
        adam_load<kState>(rv[i], t.v[k], at[i], whole[i], n);
        if constexpr (P == kAdamBf16)
            adam_load<2>(rp[i], t.param[k], at[i], whole[i], n);
        else
            adam_load<4>(rp[i], P == kAdamMaster ? t.master[k] : t.param[k], at[i], whole[i], n);
    }
    const int64_t block = first / kAdamBlock;   // (E4M3: first is a multiple)
    const float sm = E4M3 ? t.m_scale[k][block] : 0.0f, sv = E4M3 ? t.v_scale[k][block] : 0.0f;
    const float decay = -j.lr * t.decay[k], nz = a.minus_zero;
    uint64_t m[2][2], root[2][2];
    float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint64_t g[2], v[2], p[2];
        if constexpr (GF32)
            adam_get_f32(rg[i], g);
        else
            adam_get_bf16(rg[i], g);
        if constexpr (E4M3) {
            adam_get_e4m3(rm[i], m[i]);
            adam_get_e4m3(rv[i], v);
        } else {
            adam_get_f32(rm[i], m[i]);
            adam_get_f32(rv[i], v);
        }
        if constexpr (P == kAdamBf16)
            adam_get_bf16(rp[i], p);
        else
            adam_get_f32(rp[i], p);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if constexpr (E4M3) {
                m[i][e] = f2_mul(m[i][e], f2(sm, sm));
                v[e] = f2_mul(v[e], f2(sv, sv));
                v[e] = f2_mul(v[e], v[e]);
            }
            const uint64_t h = f2_mul(g[e], f2(j.clip, j.clip));
            m[i][e] = f2_add(adam_product(m[i][e], f2(a.b1, a.b1), nz), adam_product(h, f2(a.one_b1, a.one_b1), nz));
            v[e] = f2_add(adam_product(v[e], f2(a.b2, a.b2), nz),
                          adam_product(f2_mul(h, h), f2(a.one_b2, a.one_b2), nz));
            const float2 w = f2_get(v[e]);
            root[i][e] = f2(__fsqrt_rn(w.x), __fsqrt_rn(w.y));
            const float2 d = f2_get(f2_fma(root[i][e], f2(j.c2, j.c2), f2(a.eps, a.eps)));
            p[e] = f2_fma(f2_mul(m[i][e], f2(-j.rate, -j.rate)), f2(adam_rcp(d.x), adam_rcp(d.y)),
                          f2_fma(p[e], f2(decay, decay), p[e]));
            if constexpr (E4M3) {
                const float2 x = f2_get(m[i][e]), y = f2_get(root[i][e]);
                top_m = adam_max(top_m, x.x, x.y);
                top_v = adam_max(top_v, y.x, y.y);
            }
        }
        if constexpr (P == kAdamMaster) adam_put_f32(t.master[k], at[i], whole[i], n, p);
        if constexpr (P == kAdamF32)
            adam_put_f32(t.param[k], at[i], whole[i], n, p);
        else
            adam_put_bf16(t.param[k], at[i], whole[i], n, p);
        if constexpr (!E4M3) {
            adam_put_f32(t.m[k], at[i], whole[i], n, m[i]);
            adam_put_f32(t.v[k], at[i], whole[i], n, v);
        }
    }
    if constexpr (E4M3) {
        // elements behind the tensor's end are zeros here; odd lanes scale v, even ones m
        const uint32_t um = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top_m));
        const uint32_t uv = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top_v));
        float inv, scale;
        adam_scale(lane & 1 ? uv : um, inv, scale);
        const float im = __shfl_sync(0xFFFFFFFFu, inv, 0), iv = __shfl_sync(0xFFFFFFFFu, inv, 1);
        float xm[2][4], xv[2][4], low_m = 1.0f, low_v = 1.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 x = f2_get(adam_product(m[i][e], f2(im, im), nz)), y = f2_get(adam_product(root[i][e], f2(iv, iv), nz));
                xm[i][2 * e] = x.x, xm[i][2 * e + 1] = x.y;
                xv[i][2 * e] = y.x, xv[i][2 * e + 1] = y.y;
                low_m = adam_min(low_m, x.x, x.y);
                low_v = adam_min(low_v, y.x, y.y);
            }
        }
        const bool small_m = __any_sync(0xFFFFFFFFu, !(low_m >= 0x1p-6f)), small_v = __any_sync(0xFFFFFFFFu, !(low_v >= 0x1p-6f));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t group = (uint64_t)at[i] >> 2;
            uint4 w = make_uint4((uint32_t)group, (uint32_t)(group >> 32), (uint32_t)t.id[k], j.step);
#pragma unroll
            for (int r = 0; r < 10; ++r) w = philox_round(w, make_uint2(a.key0[r], a.key1[r]));
            AdamRaw q;
            q.w[0] = adam_round<false>(xm[i], small_m, w);
            adam_store<1>(t.m[k], at[i], whole[i], n, q);
            q.w[0] = adam_round<true>(xv[i], small_v, w);
            adam_store<1>(t.v[k], at[i], whole[i], n, q);
        }
        if (lane < 2) put(lane ? t.v_scale[k] : t.m_scale[k], block, (n + kAdamBlock - 1) / kAdamBlock, scale);
    }
}

// Blocks an SM, 411M elements: 8 bits 4 1446 us, 5 1206 (4 bytes of spills with masters), 6 1275 (more); fp32 2 1824, 3
// 1855, 4 1847.
template <int N, bool E4M3, AdamParam P, bool GF32>
__global__ void __launch_bounds__(kAdamThreads, E4M3 ? 5 : 2) adamw_kernel(const __grid_constant__ AdamTable<N> t,
                                                                const __grid_constant__ AdamArgs a) {
    grid_dependency();
    __shared__ float corr[2];
    AdamStep j;
    j.lr = *a.lr;
    j.clip = 1.0f;
    const int64_t step = *a.step;
    if (a.norm) {
        const float n = *a.norm, q = a.max_norm / (n + 1e-6f);
        if (!(fabsf(n) < INFINITY)) return;   // all of the grid: nothing is changed
        j.clip = q > 1.0f ? 1.0f : q;
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
    j.rate = j.lr * corr[0] * a.unit;
    j.c2 = corr[1] * a.unit;
    j.step = (uint32_t)step;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);   // the same in all lanes
    int k = 0, end = 0;   // the current tensor, and the chunk behind its last
    for (int chunk = blockIdx.x; chunk < t.first[t.count]; chunk += gridDim.x) {
        if (chunk >= end) {
            k = 0;
            int last = t.count - 1;
            while (k < last) {
                const int mid = (k + last + 1) >> 1;
                if (t.first[mid] <= chunk)
                    k = mid;
                else
                    last = mid - 1;
            }
            end = t.first[k + 1];
        }
        const int flags = t.flags[k];
        const int64_t first = (int64_t)(chunk - t.first[k]) * kAdamChunk + warp * kAdamBlock - flags / kAdamHead;
        if (first >= t.numel[k]) continue;
        if ((flags & kAdamVectors) && first >= 0 && first + kAdamBlock <= t.numel[k])
            adam_step<N, E4M3, P, GF32, true>(t, k, first, a, j, lane);
        else
            adam_step<N, E4M3, P, GF32, false>(t, k, first, a, j, lane);
    }
}

}  // namespace qt2
