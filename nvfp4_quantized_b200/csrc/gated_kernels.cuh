// gated_kernels.cuh -- the gated feed-forward product on NVFP4 operands, and its backward pass.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u                                    (forward)
//   dh = dy Wd, dg = dh u act'(g), du = dh act(g), h = act(g) u again        (backward)
//
// with act(x) = x s: s = 1 / (1 + exp(-x)) for SiLU, 1 / (1 + exp(-2 z)) for GELU's tanh form,
// z = sqrt(2/pi) (x + 0.044715 x^3), and act'(x) = s + x s (1 - s) (d/dx of the exponent, sign turned).
//
// Both are the block-scaled product of a pair of SMs (256 rows, tcgen05.mma.cta_group::2, operands by
// TMA, fp32 sums in tensor memory) with an epilogue of their own:
//   forward   a pair's 256 columns of B are 128 rows of Wg, in the first SM's shared memory, and the
//             same 128 rows of Wu, in the second's.  Every thread then finds g and u of the same
//             elements in its own TMEM lane, 128 columns apart, and x is read once for both.
//   backward  dh stays in tensor memory: the epilogue reads g and u, and writes dg, du and h.
// Rows and columns come in 128s; a tile's second half may lie behind the end (TMA fills it with zeros,
// codes and scales, and nothing of it is stored).
//
// Roles, per CTA, persistent over the tiles (K = 256 a stage):
//   warp 0        producer: a stage's scale atoms on one barrier, then its codes on another.
//   warp 1        leader: issues the MMAs; both: allocate and free tensor memory.
//   warp 2        leader: copies the scale atoms into the tensor memory of both SMs.
//   warps 4...    epilogue: warp w has TMEM lanes 32 (w % 4) on and its share of the columns; all its sums go to
//                 registers, then the accumulator is free for the next tile's MMAs.  Backward each warp loads its own
//                 pieces of gate and up by TMA ahead of their use.
// Every wait is bounded; after a timeout the leader drains what was issued, both CTAs meet, and TMEM is
// freed.
//
// 16384 x 4096 x 14336: forward, gate and up kept, 0.99 to 1.03 ms (3.8 PFLOP/s; cold and alone 4.5), not kept 0.85 ms,
// backward 0.74 to 0.77 ms (without its stores 0.59, without its loads 0.65, without the MMAs 0.67).  Memory alone
// would take 0.23 and 0.37 ms, the MMAs at four times the measured bf16 rate (6.6 PFLOP/s) 0.58 and 0.29.  Nothing is
// full: a pair streams 1.2 MB from L2 for a tile of K = 4096, 8.9 GB forward (8.7 TB/s, where the linears' GEMM gets
// 13.8) and 4.5 GB backward beside gate, up and three outputs; the tensor pipe is 61% and 39% active.  There is one
// accumulator, so the MMAs wait while a tile's sums are read, and backward a warp's load, arithmetic and stores of a
// piece come one after the other.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"
#include "qt2_pair.cuh"
#include "vec_device.cuh"

namespace qt2 {

template <bool BWD>
struct GatedCfg {
    static constexpr int kStages = BWD ? 4 : 5;
    static constexpr int kEpiWarp0 = 4;
    static constexpr int kEpiWarps = 8;
    static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
    static constexpr int kRegs = 168, kRegsOthers = 40, kRegsEpi = 232;   // a thread, at launch and (backward) then
    static constexpr int kA = 128 * 128;          // own 128 rows, K = 256
    static constexpr int kB = 128 * 128;          // own half of B's 256 rows
    static constexpr int kSfa = 4 * 512;          // 4 k-blocks x one 512-byte atom
    static constexpr int kSfb = 2 * 4 * 512;      // of all of B's rows
    static constexpr int kStageBytes = kA + kB + kSfa + kSfb;
    // what an epilogue warp has of shared memory: 32 rows x 64 columns of bf16, backward of gate and of up
    static constexpr int kPiece = 32 * 64 * 2;
    static constexpr int kOwnBytes = BWD ? 2 * kPiece : kPiece;
    static constexpr int kBars = 4 * kStages + 2 + (BWD ? kEpiWarps : 0);
    static constexpr int kSmemBytes = kStages * kStageBytes + kEpiWarps * kOwnBytes + 1024 + 512;
    static constexpr int kTmemCols = 512;         // accumulator 256 + 5 scale regions x 48
    static constexpr int kSfRegionCols = 48;
    // E2M1 x E2M1, UE4M3 scales, K-major A and B, M = 256 (pair), N = 256
    static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | (32u << 17) | (16u << 24);
    static_assert(kStageBytes % 1024 == 0, "stage alignment");
    static_assert(256 + kStages * kSfRegionCols <= kTmemCols, "TMEM columns");
    static_assert(8 * kBars + 8 <= 512, "barriers");
};

// b and sfb: gate and up (forward); the down projection in the first (backward).
struct GatedMaps {
    CUtensorMap a, b[2], sfa, sfb[2];
    CUtensorMap gate, up;   // backward
};

struct GatedArgs {
    const float *ga, *gb[2];      // tensor scales of a and of the one or two b
    float alpha;
    int M, F, K;                  // multiples of 128
    int group_m;                  // rows of tiles that are run through together
    __nv_bfloat16 *gate, *up;     // forward: written, or both null; backward: read
    int64_t ldgu;
    __nv_bfloat16 *dgate, *dup;   // backward
    int64_t lddgu;
    __nv_bfloat16 *h;             // backward: may be null
    int64_t ldh;
};

// act(x) = x s of two elements, and (SLOPE) its derivative.  exp overflows to inf, and s is 0, where x is far below
// zero.  GELU's exponent is that of x or, further than 11 from zero, of 11: 2^162 and 2^-162 there, s is 0 or 1 as it
// is from 10.01 on.  What multiplies s is x itself, so that a NaN stays one and -inf becomes one (-inf * 0).
template <int ACT, bool SLOPE>
__device__ __forceinline__ uint64_t gated_act(uint64_t x, uint64_t &slope) {
    constexpr float kLog2e = 1.4426950408889634f, c = 1.5957691216057308f, d = 0.044715f;   // c: 2 sqrt(2/pi)
    const uint64_t one = f2(1.0f, 1.0f);
    uint64_t t, rise = one;   // the exponent of s (in base 2, sign turned), and its derivative
    if constexpr (ACT == QT2_ACT_SILU) {
        t = f2_mul(x, f2(-kLog2e, -kLog2e));
    } else {
        const float2 y = f2_get(x);
        const uint64_t b = f2(fminf(fmaxf(y.x, -11.0f), 11.0f), fminf(fmaxf(y.y, -11.0f), 11.0f));
        const uint64_t q = f2_mul(b, b);
        t = f2_mul(f2_mul(b, f2(-c * kLog2e, -c * kLog2e)), f2_fma(q, f2(d, d), one));
        rise = f2_fma(q, f2(3 * c * d, 3 * c * d), f2(c, c));
    }
    const float2 e = f2_get(t);
    float ex, ey, sx, sy;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ex) : "f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ey) : "f"(e.y));
    const float2 n = f2_get(f2_add(f2(ex, ey), one));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(sx) : "f"(n.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(sy) : "f"(n.y));
    const uint64_t s = f2(sx, sy);
    const uint64_t xs = f2_mul(x, s);
    if constexpr (SLOPE) {   // s + x s (1 - s) rise
        const uint64_t t2 = f2_mul(xs, f2_fma(s, f2(-1.0f, -1.0f), one));
        slope = ACT == QT2_ACT_SILU ? f2_add(t2, s) : f2_fma(t2, rise, s);
    }
    return xs;
}
__device__ __forceinline__ uint32_t gated_bits(uint64_t v) {
    const float2 p = f2_get(v);
    return bf16_pair(p.x, p.y);
}

// A piece lies in shared memory in rows of 128 bytes whose 16-byte parts are permuted (part ^ row % 8), as TMA loads
// them with the 128-byte swizzle: a warp meets in no bank, whether each lane has a row or eight lanes share one.
// Columns [16 i, 16 i + 16) of this lane's row:
__device__ __forceinline__ void piece_get(const uint8_t *piece, int lane, int i, uint32_t (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint4 q = *reinterpret_cast<const uint4 *>(piece + lane * 128 + (((2 * i + k) ^ (lane & 7)) << 4));
        v[4 * k] = q.x; v[4 * k + 1] = q.y; v[4 * k + 2] = q.z; v[4 * k + 3] = q.w;
    }
}
__device__ __forceinline__ void piece_put(uint8_t *piece, int lane, int i, const uint32_t *v) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
        *reinterpret_cast<uint4 *>(piece + lane * 128 + (((2 * i + k) ^ (lane & 7)) << 4)) =
            make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
}
// The piece to 32 rows of a matrix, whole 128-byte lines at a time, whatever the rows' alignment.  (Each lane along its
// own row, 32 bytes at a time: forward 32768 x 2048 x 5632 484 us instead of 465, 604 where rows start on 16 bytes
// only, though 16384 x 4096 x 14336 971 instead of 1009; backward 843 instead of 824.)
__device__ __forceinline__ void piece_store(const uint8_t *piece, int lane, __nv_bfloat16 *to, int64_t ld, const void *base,
                                            uint64_t extent) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + (lane >> 3), part = lane & 7;
        __nv_bfloat16 *const p = to + row * ld + part * 8;
        const uint4 q = *reinterpret_cast<const uint4 *>(piece + row * 128 + ((part ^ (row & 7)) << 4));
        if (QT2_STORE_OK(p, 16, base, extent)) *reinterpret_cast<uint4 *>(p) = q;
    }
    __syncwarp();
}

// 64 columns of h, gate and up from their sums: v[0..63] and v[64..127].
template <int ACT>
__device__ __forceinline__ void gated_forward(const GatedArgs &a, const uint32_t (&v)[128], uint8_t *piece, int lane,
                                              int64_t row, int64_t col, float sg, float su) {
    const uint64_t hs = ((uint64_t)(a.M - 1) * a.ldh + a.F) * 2, gs = ((uint64_t)(a.M - 1) * a.ldgu + a.F) * 2;
    uint32_t pg[32], pu[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t ph[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int j = 16 * i + 2 * k;
            const uint64_t g = f2_mul(f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2(sg, sg));
            const uint64_t u = f2_mul(f2(__uint_as_float(v[64 + j]), __uint_as_float(v[65 + j])), f2(su, su));
            uint64_t none;
            ph[k] = gated_bits(f2_mul(gated_act<ACT, false>(g, none), u));
            pg[8 * i + k] = gated_bits(g);
            pu[8 * i + k] = gated_bits(u);
        }
        piece_put(piece, lane, i, ph);
    }
    piece_store(piece, lane, a.h + row * a.ldh + col, a.ldh, a.h, hs);
    if (!a.gate) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) piece_put(piece, lane, i, &pg[8 * i]);
    piece_store(piece, lane, a.gate + row * a.ldgu + col, a.ldgu, a.gate, gs);
#pragma unroll
    for (int i = 0; i < 4; ++i) piece_put(piece, lane, i, &pu[8 * i]);
    piece_store(piece, lane, a.up + row * a.ldgu + col, a.ldgu, a.up, gs);
}

// 64 columns of dgate, dup and h from the sums of dh (v) and the pieces of gate and up, which are overwritten.
template <int ACT>
__device__ __forceinline__ void gated_backward(const GatedArgs &a, const uint32_t *v, uint8_t *piece, int lane, int64_t row,
                                               int64_t col, float sc) {
    const uint64_t hs = ((uint64_t)(a.M - 1) * a.ldh + a.F) * 2, ds = ((uint64_t)(a.M - 1) * a.lddgu + a.F) * 2;
    uint8_t *const piece_u = piece + GatedCfg<true>::kPiece;
    uint32_t ph[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t pg[8], pu[8];
        piece_get(piece, lane, i, pg);
        piece_get(piece_u, lane, i, pu);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint64_t g = f2(bf16_lo(pg[k]), bf16_hi(pg[k])), u = f2(bf16_lo(pu[k]), bf16_hi(pu[k]));
            const int j = 16 * i + 2 * k;
            const uint64_t dh = f2_mul(f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f2(sc, sc));
            uint64_t slope;
            const uint64_t act = gated_act<ACT, true>(g, slope);
            pg[k] = gated_bits(f2_mul(f2_mul(dh, u), slope));
            pu[k] = gated_bits(f2_mul(dh, act));
            ph[8 * i + k] = gated_bits(f2_mul(act, u));
        }
        piece_put(piece, lane, i, pg);
        piece_put(piece_u, lane, i, pu);
    }
    piece_store(piece, lane, a.dgate + row * a.lddgu + col, a.lddgu, a.dgate, ds);
    piece_store(piece_u, lane, a.dup + row * a.lddgu + col, a.lddgu, a.dup, ds);
    if (!a.h) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) piece_put(piece, lane, i, &ph[8 * i]);
    piece_store(piece, lane, a.h + row * a.ldh + col, a.ldh, a.h, hs);
}

template <bool BWD, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GatedCfg<BWD>::kThreads, 1)
    gated_pair_kernel(const __grid_constant__ GatedMaps maps, const __grid_constant__ GatedArgs a) {
    using Cfg = GatedCfg<BWD>;
    constexpr int S = Cfg::kStages;
    constexpr int kCols = BWD ? 256 : 128;   // of F a tile
    extern __shared__ __align__(1024) uint8_t smem_dyn[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    uint8_t *const pieces = base + S * Cfg::kStageBytes;   // of the epilogue warps
    // barriers: full[S] sftm[S] empty[S] acc_full acc_empty sfull[S], backward piece[warp]
    uint64_t *bars = reinterpret_cast<uint64_t *>(pieces + Cfg::kEpiWarps * Cfg::kOwnBytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Cfg::kBars);

    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_pm = (a.M + 255) >> 8, num_pn = (a.F + kCols - 1) / kCols, tiles = num_pm * num_pn;
    const int cluster_id = blockIdx.x >> 1, num_clusters = gridDim.x >> 1;
    const int nkb = a.K >> 6, nks = (nkb + 3) >> 2;
    const int my_tiles = tiles > cluster_id ? (tiles - 1 - cluster_id) / num_clusters + 1 : 0;
    const int total = my_tiles * nks;   // stages this pair runs
    const uint32_t full0 = smem_u32(bars), sftm0 = smem_u32(bars + S), empty0 = smem_u32(bars + 2 * S);
    const uint32_t acc_full = smem_u32(bars + 3 * S), acc_empty = acc_full + 8;
    const uint32_t sfull0 = smem_u32(bars + 3 * S + 2);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);    // codes: the leader's producer (expects both SMs' bytes)
            mbar_init(sfull0 + 8 * s, 1);   // scale atoms: likewise
            mbar_init(sftm0 + 8 * s, 1);    // the scale copier's commit
            mbar_init(empty0 + 8 * s, 1);   // the MMA issuer's commit
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 2 * Cfg::kEpiWarps);
        if (BWD)
            for (int i = 0; i < Cfg::kEpiWarps; ++i) mbar_init(sfull0 + 8 * (S + i), 1);   // the warp's own loads
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), Cfg::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();   // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();

    // Tiles run over group_m rows of tiles first, then over F: those in flight share their operands' rows.
    auto tile_coords = [&](int tile, int &pm, int &pn) {
        const int group = tile / (a.group_m * num_pn), first = group * a.group_m;
        const int rows = min(a.group_m, num_pm - first), r = tile - first * num_pn;
        pn = r / rows;
        pm = first + r - pn * rows;
    };

    // Backward the epilogue's warpgroups take registers over from the others', so that the arithmetic of 64 columns
    // overlaps beside the 128 sums (16384 x 4096 x 14336: 168 a thread 824 us, 216 816, 224 775, 232 750; 52 bytes are
    // still spilled with GELU, 60 with SiLU).  Forward 168 hold it all.
    static_assert(128 * Cfg::kRegsOthers + 32 * Cfg::kEpiWarps * Cfg::kRegsEpi <= Cfg::kRegs * Cfg::kThreads, "register split");

    int issued = 0, mma_done = 0, copied = 0;   // stages whose loads, MMAs and scale copies were issued
    if (BWD && warp < Cfg::kEpiWarp0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsOthers));
    if (warp == 0) {
        // -------------------------------------------------------------- producer (both CTAs)
        if (elect_one()) {
            prefetch_tmap(&maps.a);
            prefetch_tmap(&maps.sfa);
            for (int i = 0; i < (BWD ? 1 : 2); ++i) {
                prefetch_tmap(&maps.b[i]);
                prefetch_tmap(&maps.sfb[i]);
            }
        }
        __syncwarp();
        const uint32_t full_leader0 = mapa_shared(full0, 0), sfull_leader0 = mapa_shared(sfull0, 0);
        // B's own half: gate rows in the leader, up rows in the other; backward the halves of 256 rows
        const CUtensorMap *const tmB = &maps.b[BWD ? 0 : rank];
        int it = 0;
        for (int t = 0; t < my_tiles && it == t * nks; ++t) {
            int pm, pn;
            tile_coords(cluster_id + t * num_clusters, pm, pn);
            for (int ks = 0; ks < nks; ++ks) {
                const int s = it % S;
                if (it >= S && !mbar_wait_warp(empty0 + 8 * s, ((it / S) & 1) ^ 1)) break;
                const uint32_t st = smem_u32(base + s * Cfg::kStageBytes);
                if (elect_one()) {
                    const uint32_t sb = sfull_leader0 + 8 * s, fb = full_leader0 + 8 * s;
                    if (leader) {
                        mbar_arrive_expect_tx(sfull0 + 8 * s, 2 * (Cfg::kSfa + Cfg::kSfb));
                        mbar_arrive_expect_tx(full0 + 8 * s, 2 * (Cfg::kA + Cfg::kB));
                    }
                    const uint32_t sfa = st + Cfg::kA + Cfg::kB, sfb = sfa + Cfg::kSfa;
                    tma_load_2d_pair(sfa, &maps.sfa, ks * 256, pm * 2 + (int)rank, sb);
                    if constexpr (BWD) {
                        tma_load_2d_pair(sfb, &maps.sfb[0], ks * 256, pn * 2, sb);
                    } else {
                        tma_load_2d_pair(sfb, &maps.sfb[0], ks * 256, pn, sb);
                        tma_load_2d_pair(sfb + Cfg::kSfb / 2, &maps.sfb[1], ks * 256, pn, sb);
                    }
                    tma_load_2d_pair(st, &maps.a, ks * 128, pm * 256 + (int)rank * 128, fb);
                    tma_load_2d_pair(st + Cfg::kA, tmB, ks * 128, BWD ? pn * 256 + (int)rank * 128 : pn * 128, fb);
                }
                __syncwarp();
                issued = ++it;
            }
        }
    } else if (warp == 1 && leader) {
        // -------------------------------------------------------------- MMA issuer (leader)
        int it = 0;
        bool ok = true;
        for (int t = 0; t < my_tiles && ok; ++t) {
            if (t > 0 && !mbar_wait_warp(acc_empty, (t - 1) & 1)) break;
            tc_fence_after();
            for (int ks = 0; ks < nks; ++ks, ++it) {
                const int s = it % S;
                const uint32_t par = (it / S) & 1;
                if (!mbar_wait_warp(full0 + 8 * s, par) || !mbar_wait_warp(sftm0 + 8 * s, par)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int nk = min(4, nkb - ks * 4);
                const uint32_t st = smem_u32(base + s * Cfg::kStageBytes);
                const uint32_t t_sf = tmem + 256 + Cfg::kSfRegionCols * s;
                if (elect_one()) {
                    for (int kk = 0; kk < nk; ++kk) {
                        const uint64_t adesc = make_smem_desc(st + 32 * kk, 16, 1024, 2);
                        const uint64_t bdesc = make_smem_desc(st + Cfg::kA + 32 * kk, 16, 1024, 2);
                        tc_mma_pair_nvfp4(tmem, adesc, bdesc, Cfg::kIdesc, t_sf + 4 * kk, t_sf + 16 + 8 * kk,
                                          (ks | kk) != 0);
                    }
                    tc_commit_pair_both(empty0 + 8 * s);
                }
                __syncwarp();
                mma_done = it + 1;
            }
            if (ok) {
                if (elect_one()) tc_commit_pair_both(acc_full);
                __syncwarp();
            }
        }
    } else if (warp == 2 && leader) {
        // -------------------------------------------------------------- scale copier (leader)
        // The stage's scales landed, so the MMAs that last used its scale region completed.
        for (int j = 0; j < total; ++j) {
            const int s = j % S;
            if (!mbar_wait_warp(sfull0 + 8 * s, (j / S) & 1)) break;
            tc_fence_after();
            const int nk = min(4, nkb - (j % nks) * 4);
            const uint32_t sfa = smem_u32(base + s * Cfg::kStageBytes + Cfg::kA + Cfg::kB), sfb = sfa + Cfg::kSfa;
            const uint32_t t_sf = tmem + 256 + Cfg::kSfRegionCols * s;
            if (elect_one()) {
                for (int kk = 0; kk < nk; ++kk) {
                    tc_cp_pair_32x128b_warpx4(t_sf + 4 * kk, make_smem_desc(sfa + 512 * kk, 0, 128, 0));
                    tc_cp_pair_32x128b_warpx4(t_sf + 16 + 8 * kk, make_smem_desc(sfb + 512 * kk, 0, 128, 0));
                    tc_cp_pair_32x128b_warpx4(t_sf + 20 + 8 * kk, make_smem_desc(sfb + 2048 + 512 * kk, 0, 128, 0));
                }
                tc_commit_pair_leader(sftm0 + 8 * s);
            }
            __syncwarp();
            copied = j + 1;
        }
    } else if (warp >= Cfg::kEpiWarp0) {
        if (BWD) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
        // -------------------------------------------------------------- epilogue (both CTAs)
        constexpr int kOwn = kCols / 2;   // columns of F that a warp has of a tile
        const int quad = warp & 3, part = (warp - Cfg::kEpiWarp0) >> 2, ew = warp - Cfg::kEpiWarp0;
        const uint32_t acc_empty_leader = mapa_shared(acc_empty, 0);
        const float sc0 = a.alpha * *a.ga * *a.gb[0], sc1 = BWD ? 0.0f : a.alpha * *a.ga * *a.gb[1];
        uint8_t *const piece = pieces + ew * Cfg::kOwnBytes;
        // Backward: the warp's pieces of gate and up, two a tile.  One is loaded as soon as the one before it has left.
        const uint32_t piece_bar = sfull0 + 8 * (S + ew);
        int loads = 0, used = 0;
        auto piece_at = [&](int j, int &x, int &y) {
            int pm, pn;
            tile_coords(cluster_id + (j >> 1) * num_clusters, pm, pn);
            y = pm * 256 + (int)rank * 128 + quad * 32;
            x = pn * kCols + part * kOwn + (j & 1) * 64;
        };
        auto load_piece = [&] {   // by one lane of the converged warp
            if (loads == 2 * my_tiles) return;
            int x, y;
            piece_at(loads, x, y);
            if (elect_one()) {
                const uint32_t to = smem_u32(piece);
                mbar_arrive_expect_tx(piece_bar, 2 * Cfg::kPiece);
                tma_load_2d(to, &maps.gate, x, y, piece_bar);
                tma_load_2d(to + Cfg::kPiece, &maps.up, x, y, piece_bar);
            }
            __syncwarp();
            ++loads;
        };
        if constexpr (BWD) load_piece();
        for (int t = 0; t < my_tiles; ++t) {
            if (!mbar_wait_warp(acc_full, t & 1)) break;
            tc_fence_after();
            int pm, pn;
            tile_coords(cluster_id + t * num_clusters, pm, pn);
            const int64_t row = (int64_t)pm * 256 + rank * 128 + quad * 32;   // the warp's first
            const int64_t col = (int64_t)pn * kCols + part * kOwn;
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + part * kOwn;
            const bool inside = row < a.M && col < a.F;   // M and F are multiples of 128: all of the warp's or nothing
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 128; c += 16)   // forward: 64 columns of gate, and of up 128 columns on
                tmem_ld_32x32b_x16(taddr + c + (!BWD && c >= 64 ? 64 : 0), *reinterpret_cast<uint32_t(*)[16]>(&v[c]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(acc_empty_leader);
            if constexpr (!BWD) {
                if (inside) gated_forward<ACT>(a, v, piece, lane, row, col, sc0, sc1);
            } else {
                bool ok = true;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ok = ok && mbar_wait_warp(piece_bar, used & 1);
                    if (!ok) continue;
                    ++used;
                    if (inside) gated_backward<ACT>(a, &v[64 * i], piece, lane, row, col + 64 * i, sc0);
                    fence_proxy_async();   // this lane's accesses to the piece come before the load's
                    __syncwarp();
                    load_piece();
                }
                if (!ok) break;
            }
        }
        // after a timeout the warp's own load is waited for
        if constexpr (BWD)
            for (; used < loads; ++used) mbar_wait_warp(piece_bar, used & 1);
    }
    // Every role ends converged.  Only after a timeout can work still be in flight: the leader
    // waits (bounded) for the loads it issued past the last consumed stage and for the last
    // issued MMAs and copies, then both CTAs meet before TMEM is freed.
    __shared__ int consumed, issued_here;
    if (warp == 1 && leader && lane == 0) consumed = mma_done;
    if (warp == 0 && lane == 0) issued_here = issued;
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (leader && warp == 0 && lane == 0) {
        const int peer = (int)ld_shared_cluster_u32(mapa_shared(smem_u32(&issued_here), 1));
        const int last = max(issued, peer);
        for (int it = consumed; it < last; ++it) {
            mbar_wait(full0 + 8 * (it % S), (it / S) & 1);
            mbar_wait(sfull0 + 8 * (it % S), (it / S) & 1);
        }
    }
    if (leader && warp == 1 && lane == 0 && mma_done > 0) {
        const int it = mma_done - 1;
        mbar_wait(empty0 + 8 * (it % S), (it / S) & 1);
    }
    if (leader && warp == 2 && lane == 0 && copied > 0) {
        const int j = copied - 1;
        mbar_wait(sftm0 + 8 * (j % S), (j / S) & 1);
    }
    cluster_sync_all();   // no SM frees TMEM or exits while its pair may still touch it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, Cfg::kTmemCols);
}

}  // namespace qt2
