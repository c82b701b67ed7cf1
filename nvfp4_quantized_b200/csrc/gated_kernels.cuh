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
// Roles, per CTA of 384 threads, persistent over the tiles (K = 256 a stage, a ring of 5):
//   warp 0        producer: a stage's scale atoms on one barrier, then its codes on another.
//   warp 1        leader: issues the MMAs; both: allocate and free tensor memory.
//   warp 2        leader: copies the scale atoms into the tensor memory of both SMs.
//   warps 4..11   epilogue: warp w has TMEM lanes 32 (w % 4) on and half of the columns; all its sums go to
//                 registers, then the accumulator is free for the next tile's MMAs.
// Every wait is bounded; after a timeout the leader drains what was issued, both CTAs meet, and TMEM is
// freed.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"
#include "qt2_pair.cuh"
#include "vec_device.cuh"

namespace qt2 {

struct GatedCfg {
    static constexpr int kStages = 5;
    static constexpr int kThreads = 384;
    static constexpr int kEpiWarp0 = 4;
    static constexpr int kEpiWarps = 8;
    static constexpr int kA = 128 * 128;          // own 128 rows, K = 256
    static constexpr int kB = 128 * 128;          // own half of B's 256 rows
    static constexpr int kSfa = 4 * 512;          // 4 k-blocks x one 512-byte atom
    static constexpr int kSfb = 2 * 4 * 512;      // of all of B's rows
    static constexpr int kStageBytes = kA + kB + kSfa + kSfb;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024 + 512;
    static constexpr int kTmemCols = 512;         // accumulator 256 + 5 scale regions x 48
    static constexpr int kSfRegionCols = 48;
    // E2M1 x E2M1, UE4M3 scales, K-major A and B, M = 256 (pair), N = 256
    static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | (32u << 17) | (16u << 24);
};
static_assert(GatedCfg::kStageBytes % 1024 == 0, "stage alignment");
static_assert(256 + GatedCfg::kStages * GatedCfg::kSfRegionCols <= GatedCfg::kTmemCols, "TMEM columns");

// b and sfb: gate and up (forward); the down projection in the first (backward).
struct GatedMaps {
    CUtensorMap a, b[2], sfa, sfb[2];
};

struct GatedArgs {
    const float *ga, *gb[2];      // tensor scales of a and of the one or two b
    float alpha;
    int M, F, K;                  // multiples of 128
    int m_fast;                   // tiles run over M first
    int wide;                     // every array's rows start on 32 bytes
    __nv_bfloat16 *gate, *up;     // forward: written, or both null; backward: read
    int64_t ldgu;
    __nv_bfloat16 *dgate, *dup;   // backward
    int64_t lddgu;
    __nv_bfloat16 *h;             // backward: may be null
    int64_t ldh;
};

__device__ __forceinline__ float gated_exp(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// s of act(x) = x s, and its derivative.  exp overflows to inf and s to 0 where x is far below zero.
template <int ACT>
__device__ __forceinline__ float gated_sigmoid(float x, float &rise) {
    if constexpr (ACT == QT2_ACT_SILU) {
        const float s = __fdividef(1.0f, 1.0f + gated_exp(-x));
        rise = s * (1.0f - s);
        return s;
    } else {
        constexpr float c = 1.5957691216057308f;   // 2 sqrt(2/pi)
        const float b = fminf(fmaxf(x, -10.0f), 10.0f), q = b * b;   // further out s is 0 or 1
        const float s = __fdividef(1.0f, 1.0f + gated_exp(-c * b * fmaf(0.044715f, q, 1.0f)));
        rise = s * (1.0f - s) * c * fmaf(3.0f * 0.044715f, q, 1.0f);
        return s;
    }
}

// 16 bf16 of a row; 16-byte aligned, or (wide) 32.
__device__ __forceinline__ void gated_store(__nv_bfloat16 *p, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        st_global_v8(p, v);
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
__device__ __forceinline__ void gated_load(const __nv_bfloat16 *p, uint32_t (&v)[8]) {
    const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// 64 columns of h from the sums of gate (v[0..63]) and up (v[64..127]).
template <int ACT>
__device__ __forceinline__ void gated_forward(const GatedArgs &a, const uint32_t (&v)[128], int64_t row, int64_t col,
                                              float sg, float su) {
    const uint64_t hs = ((uint64_t)(a.M - 1) * a.ldh + a.F) * 2, gs = ((uint64_t)(a.M - 1) * a.ldgu + a.F) * 2;
    __nv_bfloat16 *const h = a.h + row * a.ldh + col;
    __nv_bfloat16 *const gate = a.gate + row * a.ldgu + col, *const up = a.up + row * a.ldgu + col;
    if (!QT2_STORE_OK(h, 128, a.h, hs)) return;
    if (a.gate && (!QT2_STORE_OK(gate, 128, a.gate, gs) || !QT2_STORE_OK(up, 128, a.up, gs))) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t ph[8], pg[8], pu[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int j = 16 * i + 2 * k;
            const float g0 = __uint_as_float(v[j]) * sg, g1 = __uint_as_float(v[j + 1]) * sg;
            const float u0 = __uint_as_float(v[64 + j]) * su, u1 = __uint_as_float(v[65 + j]) * su;
            float r;
            ph[k] = bf16_pair(g0 * gated_sigmoid<ACT>(g0, r) * u0, g1 * gated_sigmoid<ACT>(g1, r) * u1);
            pg[k] = bf16_pair(g0, g1);
            pu[k] = bf16_pair(u0, u1);
        }
        gated_store(h + 16 * i, ph, a.wide);
        if (a.gate) {
            gated_store(gate + 16 * i, pg, a.wide);
            gated_store(up + 16 * i, pu, a.wide);
        }
    }
}

// 128 columns of dgate, dup and h from the sums of dh.
template <int ACT>
__device__ __forceinline__ void gated_backward(const GatedArgs &a, const uint32_t (&v)[128], int64_t row, int64_t col,
                                               float sc) {
    const uint64_t hs = ((uint64_t)(a.M - 1) * a.ldh + a.F) * 2, ds = ((uint64_t)(a.M - 1) * a.lddgu + a.F) * 2;
    const __nv_bfloat16 *const gate = a.gate + row * a.ldgu + col, *const up = a.up + row * a.ldgu + col;
    __nv_bfloat16 *const dg = a.dgate + row * a.lddgu + col, *const du = a.dup + row * a.lddgu + col;
    __nv_bfloat16 *const h = a.h + row * a.ldh + col;
    if (!QT2_STORE_OK(dg, 256, a.dgate, ds) || !QT2_STORE_OK(du, 256, a.dup, ds)) return;
    if (a.h && !QT2_STORE_OK(h, 256, a.h, hs)) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t pg[8], pu[8], ph[8];
        gated_load(gate + 16 * i, pg);
        gated_load(up + 16 * i, pu);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float d[2], e[2], f[2];
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const float g = o ? bf16_hi(pg[k]) : bf16_lo(pg[k]), u = o ? bf16_hi(pu[k]) : bf16_lo(pu[k]);
                const float dh = __uint_as_float(v[16 * i + 2 * k + o]) * sc;
                float rise;
                const float s = gated_sigmoid<ACT>(g, rise), act = g * s;
                const float x = ACT == QT2_ACT_SILU ? g : fminf(fmaxf(g, -10.0f), 10.0f);
                d[o] = dh * u * fmaf(x, rise, s);
                e[o] = dh * act;
                f[o] = act * u;
            }
            pg[k] = bf16_pair(d[0], d[1]);
            pu[k] = bf16_pair(e[0], e[1]);
            ph[k] = bf16_pair(f[0], f[1]);
        }
        gated_store(dg + 16 * i, pg, a.wide);
        gated_store(du + 16 * i, pu, a.wide);
        if (a.h) gated_store(h + 16 * i, ph, a.wide);
    }
}

template <bool BWD, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GatedCfg::kThreads, 1)
    gated_pair_kernel(const __grid_constant__ GatedMaps maps, const __grid_constant__ GatedArgs a) {
    using Cfg = GatedCfg;
    constexpr int S = Cfg::kStages;
    constexpr int kCols = BWD ? 256 : 128;   // of F a tile
    extern __shared__ __align__(1024) uint8_t smem_dyn[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    // barriers: full[S] sftm[S] empty[S] acc_full acc_empty sfull[S]
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + S * Cfg::kStageBytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 4 * S + 2);

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

    // With m_fast the tiles in flight cover all of a small x and a few row blocks of the weights, which
    // then stream from DRAM once; else the other way round.
    auto tile_coords = [&](int tile, int &pm, int &pn) {
        if (a.m_fast) {
            pn = tile / num_pm;
            pm = tile - pn * num_pm;
        } else {
            pm = tile / num_pn;
            pn = tile - pm * num_pn;
        }
    };

    int issued = 0, mma_done = 0, copied = 0;   // stages whose loads, MMAs and scale copies were issued
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
        // -------------------------------------------------------------- epilogue (both CTAs)
        const int quad = warp & 3, half = (warp - Cfg::kEpiWarp0) >> 2;
        const uint32_t acc_empty_leader = mapa_shared(acc_empty, 0);
        const float sc0 = a.alpha * *a.ga * *a.gb[0], sc1 = BWD ? 0.0f : a.alpha * *a.ga * *a.gb[1];
        for (int t = 0; t < my_tiles; ++t) {
            if (!mbar_wait_warp(acc_full, t & 1)) break;
            tc_fence_after();
            int pm, pn;
            tile_coords(cluster_id + t * num_clusters, pm, pn);
            const int64_t row = (int64_t)pm * 256 + rank * 128 + quad * 32 + lane;
            const int64_t col = (int64_t)pn * kCols + half * (kCols / 2);
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + half * (kCols / 2);
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 128; c += 16)   // forward: 64 columns of gate, and of up 128 columns on
                tmem_ld_32x32b_x16(taddr + c + (!BWD && c >= 64 ? 64 : 0), *reinterpret_cast<uint32_t(*)[16]>(&v[c]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(acc_empty_leader);
            if (row >= a.M || col >= a.F) continue;   // M and F are multiples of 128: all of the warp's or nothing
            if constexpr (BWD)
                gated_backward<ACT>(a, v, row, col, sc0);
            else
                gated_forward<ACT>(a, v, row, col, sc0, sc1);
        }
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
