// xent_kernels.cuh -- the head's softmax cross entropy without its logits.
//
//   l = x w^T, lse_t = log sum_v exp l_tv, loss_t = lse_t - l_t,y(t)          (forward)
//   G_tv = dloss_t (exp(l_tv - lse_t) - [v = y(t)]), dx = G w, dw = G^T x     (backward)
//
// The tensor cores take G as c_t P_tv: with q_t = 1 - exp(l_t,y(t) - lse_t), the rest of the row's
// probability, c_t = dloss_t q_t and P_tv = exp(l_tv - lse_t) / q_t, -1 at the target.  P's largest entry
// is then exact in bf16 and the others' roundings independent; c_t multiplies dx's rows in fp32, and
// x's for dw.  Rounded as it stands, G's entry at the target is off by up to 2^-8 in all of dx's row, and
// equal dloss in all rows alike.
//
// c x is the sum of two bf16 numbers (2^-16 off at most).  P is multiplied by the first.  The second
// takes part where an entry of P shows c x in full, at the targets: the tokens are sorted by the tile of
// dw that holds their target (stable: the sums' order is fixed), and a tile multiplies its tokens' second
// numbers by a matrix H of one entry a row, P's at the target: a stage or so more a tile.  Products with
// P's other entries have that entry's rounding anyway.  With the first number alone an fp32 dw was off by
// 1.6e-3 to 2.2e-3 (2-norm; 300 x 1000 x 8000 with equal dloss), and a bf16 one by 2.2e-3, of which 1.65e-3
// are its own rounding.  (P times both numbers wherever a tile and a stage of 64 tokens hold a target, which
// needs no sorting: backward 2048 x 2048 x 32000 697 us, with sorting 570, with one number 530; 8192 x 1024 x
// 1000, 5100 targets in one tile of four, 143, 130 and 92.)
//
// All three products are bf16 with fp32 sums on the tensor cores, in one persistent kernel shape
// (mm_pair_kernel): a pair of SMs forms 256x256 tiles with tcgen05.mma.cta_group::2, each SM
// holding its 128 rows of A and half of B, so that a stage of K = 64 moves 64 KB for 8.4 MFLOP.
// What differs is where the operands come from and what the epilogue does with a tile:
//   kLoss   A = x, B = w rows; the tile of logits becomes one (max, sum of exp) pair a row and
//           128 columns, and the target's logit where the tile holds it.
//   kProbs  the same tile becomes the bf16 entries of P for one piece of the vocabulary.
//           Fewer than 32 tokens (SWAP): A = w rows, B = x; a thread then holds one vocabulary entry of
//           every token.  With so few rows of x as A, every pair's loads of a stage meet in the same few
//           L2 lines (32000 x 2048: 44 us for 1 token, 38 us for 16, 32 us for 32; swapped 28, 32 and 35).
//   kGrads  jobs of both gradient products in one launch: dx (A = P, B = w with the vocabulary
//           contracted, so w is read transposed: an MN-major operand) added up over the pieces in
//           fp32, and dw (A = P transposed, B = a copy of x transposed), whose rows are complete
//           after their piece.
//
// Tensor cores bound it, and over longer times the power limit: at 2048 x 2048 x 32000 the tensor pipes
// are active for 95 / 93 / 97% of the three kernels' cycles; forward 4096 x 2048 x 50257 0.50 ms at full
// clocks (1.68 PFLOP/s), 0.59 ms under the limit.  Rows that start off 128-byte lines cost: hidden 1000
// instead of 1024 takes the forward pass at 777 tokens from 73 to 88 us, since each 128-byte row of a
// load then touches two L2 lines.
#pragma once

#include <cuda_bf16.h>

#include "qt2_device.cuh"
#include "qt2_pair.cuh"
#include "vec_device.cuh"

namespace qt2 {

// D[tmem] (+)= A[smem] x B[smem], bf16, one pair of SMs (K = 16 per instruction).
__device__ __forceinline__ void tc_mma_pair_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(d) of a difference: taken before the factor log2(e), which would round numbers as large as the
// logits (at 1e7 to halves).
__device__ __forceinline__ float exp_of(float d) { return ex2(d * 1.4426950408889634f); }

// What logits of maximum m are reduced by before exp: where m is infinite nothing (m - m is no number), so that
// exponentials of -inf add up to 0 and one of +inf to inf.
__device__ __forceinline__ float exp_ref(float m) { return fabsf(m) == INFINITY ? 0.0f : m; }

constexpr int kSwapN = 32;   // SWAP: its tiles' columns, the least that a pair's MMA takes
template <bool SWAP>
struct MmCfg {
    static constexpr int kStages = SWAP ? 11 : 7;
    static constexpr int kThreads = 384;
    static constexpr int kEpiWarp0 = 4;
    static constexpr int kEpiWarps = 8;
    static constexpr int kA = 128 * 64 * 2;   // own 128 rows of A, K = 64
    static constexpr int kN = SWAP ? kSwapN : 256;
    static constexpr int kB = kN / 2 * 64 * 2;   // own half of B's rows
    static constexpr int kStageBytes = kA + kB;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024 + 512;
    static constexpr int kTmemCols = 512;     // two 256-column accumulators
    // fp32 sums, bf16 A and B, M = 256 (pair), N = kN; bits 15 / 16: A / B is MN-major
    static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kN / 8) << 17) | (16u << 24);
    static constexpr uint32_t kIdescMnA = 1u << 15, kIdescMnB = 1u << 16;
};

enum MmMode { kLoss = 0, kProbs = 1, kGrads = 2 };

// Tensor maps: k = K-major reads (box 64 x 128 rows), mn = MN-major reads (box 64 x 64).
struct MmMaps {
    CUtensorMap x_k, w_k, p_k, x_mn, low_mn, h_mn, w_mn, p_mn;
};

// What the backward pass needs of a row: lse, 1 / q (0: no target), P's entry at the target, c.
struct __align__(16) XentRow {
    float lse, inv, at, c;
};

// Of a 256-wide tile of the vocabulary: where the tokens that have their target in it begin in sorted order, how
// many they are, and their first row of H (a multiple of kTileRows).
struct __align__(16) XentTile {
    int start, count, h, none;
};
constexpr int kTileRows = 16;   // K of one MMA: a tile's rows of H are filled up with zeros to a multiple of it

struct MmArgs {
    int T, K, V;
    int v0, vw;            // the piece: its first vocabulary entry and its width (a multiple of 256)
    const int64_t *targets;
    int64_t ignore;
    float2 *part;          // kLoss: [parts][T]
    int parts;
    const __nv_bfloat16 *x, *w;   // for the targets' logits
    int64_t ldx, ldw;
    __nv_bfloat16 *xs;     // backward, where dw is wanted: c x, zeros in rows without a target
    int64_t ldxs;
    __nv_bfloat16 *low;    // what c x's rounding to xs left over, rows in sorted order
    __nv_bfloat16 *H;      // [h_rows][256]: P's entry at the target, in column target % 256
    int64_t h_rows;
    int *count;            // [num_v + 1][words]: tokens of a tile in each 2048; then what comes before them in sorted order
    int words;
    int *pos;              // [T]: the token's place in sorted order, behind the tiles' those without a target
    XentTile *tile;        // [num_v]
    XentRow *rows;         // backward: [T]
    float *hit, *exact;    // kLoss: the target's logit as the tile has it, and formed in fp32
    __nv_bfloat16 *P;      // [T][vw]
    int num_m, num_n;      // kLoss, kProbs: tiles of the tokens and of the vocabulary
    int group_m;           // of the tokens' tiles, those that go with each tile of the vocabulary in turn
    int dx_jobs, splits, dx_m, dx_n;   // kGrads: dx's jobs come first: (split, row tile, column tile)
    int dw_jobs, lead;     // lead: dw jobs that a pair without an extra dx job is ahead
    int add;               // dx's sums hold earlier pieces
    float *acc;            // [splits][256 dx_m][256 dx_n]
    void *dw;
    int64_t lddw;
    int dw_f32, dw_wide;   // dw_wide: its rows start 32-byte aligned
};

// One job: its tile, and the stages [ks, ks + nk) of its contraction.
struct MmJob {
    int m, n, ks, nk, split;
    bool dw;
};

// The i-th job of pair c of `pairs`; false: it has no more.  Tiles go round the pairs in turn, so that
// those in flight are neighbours and share operands in L2.  kGrads: dx's jobs, which are long, go
// round first; the first dx_jobs % pairs pairs then have one more than the others, which run `lead`
// of dw's short jobs before these join in (without it a 777-token step left pairs idle for a third of
// the launch).
template <int MODE>
__device__ __forceinline__ bool mm_job(const MmArgs &a, int c, int pairs, int i, MmJob &b) {
    b.split = 0;
    b.dw = false;
    b.ks = 0;
    if (MODE != kGrads) {
        // along the tokens first, in groups of tiles: those in flight share the group's part of x and few rows of w
        int j = c + i * pairs;
        if (j >= a.num_m * a.num_n) return false;
        const int group = j / (a.group_m * a.num_n), first = group * a.group_m, rows = min(a.group_m, a.num_m - first);
        j -= first * a.num_n;
        b.n = j / rows;
        b.m = first + j - b.n * rows;
        b.nk = (a.K + 63) >> 6;
        return true;
    }
    int j = c + i * pairs;
    if (j < a.dx_jobs) {
        const int nks = a.vw >> 6, tiles = a.dx_m * a.dx_n;
        b.split = j / tiles;
        j -= b.split * tiles;
        b.m = j / a.dx_n;
        b.n = j - b.m * a.dx_n;
        const int lo = (int)((int64_t)nks * b.split / a.splits), hi = (int)((int64_t)nks * (b.split + 1) / a.splits);
        b.ks = lo;
        b.nk = hi - lo;
        return true;
    }
    const int extra = a.dx_jobs % pairs;                         // pairs with one more dx job
    const int k = i - a.dx_jobs / pairs - (c < extra ? 1 : 0);   // this pair's k-th dw job
    if (c < extra)
        j = a.lead * (pairs - extra) + k * pairs + c;
    else
        j = k < a.lead ? k * (pairs - extra) + c - extra : a.lead * (pairs - extra) + (k - a.lead) * pairs + c;
    if (j >= a.dw_jobs) return false;
    const int nn = (a.K + 255) >> 8;
    b.dw = true;
    b.m = j / nn;
    b.n = j - b.m * nn;
    b.nk = (a.T + 63) >> 6;
    return true;
}

// What a dw job's tile has behind its stages: the products with H (count 0: no dw job).
template <int MODE>
__device__ __forceinline__ XentTile mm_tile(const MmArgs &a, const MmJob &b) {
    if (MODE != kGrads || !b.dw) return {};
    return a.tile[(a.v0 >> 8) + b.m];
}

// The row's target within the vocabulary, or -1.
__device__ __forceinline__ int xent_target(const MmArgs &a, int64_t t) {
    const int64_t y = a.targets[t];
    return (y == a.ignore || y < 0 || y >= a.V) ? -1 : (int)y;
}

// The target's logit again, in fp32 with short sums, by one warp: the tensor cores' long ones lose up
// to 1.7e-5 of it (K = 4096, products of one sign), which the loss of a row that expects its target
// otherwise shows in full.
__device__ __forceinline__ float xent_exact(const MmArgs &a, int64_t t, int y, int lane) {
    const __nv_bfloat16 *x = a.x + t * a.ldx, *w = a.w + (int64_t)y * a.ldw;
    float h = 0.0f;
#pragma unroll 4
    for (int k = lane * 8; k < a.K; k += 256) {
        const uint4 u = *reinterpret_cast<const uint4 *>(x + k), v = *reinterpret_cast<const uint4 *>(w + k);
        const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
        float d = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k + 2 * e < a.K) d = fmaf(bf16_lo(uw[e]), bf16_lo(vw[e]), d);
            if (k + 2 * e + 1 < a.K) d = fmaf(bf16_hi(uw[e]), bf16_hi(vw[e]), d);
        }
        h += d;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) h += __shfl_xor_sync(0xFFFFFFFFu, h, o);
    return h;
}

// Backward, where dw is wanted: the tokens' stable order by the tile of their target (tile num_v: none), in three
// phases: a block counts 2048 tokens a tile (kCount); one block adds up the counts before each (kScan); a
// block gives its 2048 tokens their places (kRank): every warp ranks 32 tokens among themselves, then one warp
// goes over these groups in their order (2048 tokens: 13 us in all; one warp for both 20 us).  Up to 2048
// tokens: one launch.
constexpr int kSortTokens = 2048, kSortTiles = 4096;   // of a block; tiles at a time in shared memory
enum SortPhase { kCount = 1, kScan = 2, kRank = 4 };

// Exclusive sum over the block's 1024 threads of v, on top of `carry`, which gains their sum.
__device__ __forceinline__ int sort_scan(int v, int &carry, int (&sh)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();   // the last call's sums are read
    if (lane == 31) sh[warp] = s;
    __syncthreads();
    int before = lane < warp ? sh[lane] : 0, all = sh[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    }
    const int r = carry + before + s - v;
    carry += all;
    return r;
}

__global__ void __launch_bounds__(1024) xent_sort_kernel(const MmArgs a, int phases) {
    grid_dependency();
    __shared__ int n_of[kSortTiles], tile_of[kSortTokens], sh[32];
    __shared__ uint8_t rank_of[kSortTokens];   // within its 32 tokens; 128: the last of its tile there
    const int tiles = (a.V + 255) >> 8, word = blockIdx.x, tid = threadIdx.x;
    const int64_t first = (int64_t)word * kSortTokens, all = (int64_t)(tiles + 1) * a.words;
    const int tokens = (int)min((int64_t)kSortTokens, a.T - first);
    if (phases & (kCount | kRank)) {
        for (int i = tid; i < tokens; i += 1024) {
            const int y = xent_target(a, first + i);
            tile_of[i] = y < 0 ? tiles : y >> 8;
        }
    }
    if (phases & kCount) {
        for (int lo = 0; lo <= tiles; lo += kSortTiles) {
            const int n = min(kSortTiles, tiles + 1 - lo);
            for (int i = tid; i < n; i += 1024) n_of[i] = 0;
            __syncthreads();
            for (int i = tid; i < tokens; i += 1024) {
                const int k = tile_of[i] - lo;
                if (k >= 0 && k < n) atomicAdd(n_of + k, 1);   // a count: the same in any order
            }
            __syncthreads();
            for (int i = tid; i < n; i += 1024) put(a.count, (int64_t)(lo + i) * a.words + word, all, n_of[i]);
            __syncthreads();
        }
    }
    if (phases & kScan) {
        int carry = 0;
        for (int64_t i = 0; i < all; i += 1024) {
            const int64_t k = i + tid;
            const int before = sort_scan(k < all ? a.count[k] : 0, carry, sh);
            if (k < all) put(a.count, k, all, before);
        }
        __syncthreads();
        carry = 0;
        for (int i = 0; i < tiles; i += 1024) {
            const int64_t k = i + tid;
            XentTile t{};
            if (k < tiles) {
                t.start = a.count[k * a.words];
                t.count = a.count[(k + 1) * a.words] - t.start;
            }
            t.h = sort_scan((t.count + kTileRows - 1) / kTileRows * kTileRows, carry, sh);
            if (k < tiles) put(a.tile, k, (int64_t)tiles, t);
        }
        __syncthreads();
    }
    if (phases & kRank) {
        __syncthreads();
        for (int i = tid; i < kSortTokens; i += 1024) {
            const int lane = tid & 31;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, i < tokens ? tile_of[i] : -1);
            rank_of[i] = (uint8_t)(__popc(same & ((1u << lane) - 1)) | ((same >> lane) == 1 ? 128 : 0));
        }
        for (int lo = 0; lo <= tiles; lo += kSortTiles) {
            const int n = min(kSortTiles, tiles + 1 - lo);
            for (int i = tid; i < n; i += 1024) n_of[i] = a.count[(int64_t)(lo + i) * a.words + word];
            __syncthreads();
            if (tid < 32) {
                int k = -1, r = 0;
                auto fetch = [&](int i) {
                    k = i < tokens ? tile_of[i] - lo : -1;
                    r = i < tokens ? rank_of[i] : 0;
                };
                fetch(tid);
                for (int i = tid; i - tid < tokens; i += 32) {
                    const int tile = k, rank = r & 127;
                    const bool in = tile >= 0 && tile < n, last = r & 128;
                    fetch(i + 32);
                    const int at = in ? n_of[tile] + rank : 0;
                    __syncwarp();
                    if (in && last) n_of[tile] = at + 1;
                    __syncwarp();
                    if (in) put(a.pos, first + i, (int64_t)a.T, at);
                }
            }
            __syncthreads();
        }
    }
}

// Backward, before the pieces: what each row needs (XentRow), and for dw c x, what its rounding left over,
// and H's row.  A warp a row.  What a row without a target holds, inf and NaN among it, must not reach
// dw through a product with a zero of P: its copies are zero.
__global__ void __launch_bounds__(256) xent_rows_kernel(const MmArgs a, const float *lse, const float *dloss) {
    grid_dependency();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int y = xent_target(a, t);
    XentRow r{lse[t], 0.0f, 0.0f, 0.0f};
    if (y >= 0) {
        // q from the exponent's difference; at least 2^-24, what a sum of fp32 probabilities resolves
        const float q = -expm1f(xent_exact(a, t, y, lane) - r.lse), least = q < 0x1p-24f ? 0x1p-24f : q;
        r.inv = 1.0f / least;
        r.at = -(q < 0.0f ? 0.0f : q) * r.inv;
        if (q >= 0x1p-24f) r.at = -1.0f;
        r.c = dloss[t] * least;
    }
    if (lane == 0) put(a.rows, t, (int64_t)a.T, r);
    if (!a.xs) return;
    const int64_t pos = a.pos[t];
    if (y >= 0) {
        // the tile's last token fills up its rows of H
        const XentTile tile = a.tile[y >> 8];
        const int i = (int)pos - tile.start;
        const int last = i == tile.count - 1 ? (i | (kTileRows - 1)) : i;
        const __nv_bfloat16 e = __float2bfloat16_rn(r.at);
        for (int k = i; k <= last; ++k) {
            uint32_t v[4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k == i && lane * 4 + j == (y & 255) >> 1)
                    v[j] = (uint32_t)*reinterpret_cast<const uint16_t *>(&e) << (16 * (y & 1));
            __nv_bfloat16 *dst = a.H + ((int64_t)tile.h + k) * 256 + lane * 8;
            if (QT2_STORE_OK(dst, 16, a.H, a.h_rows * 512))
                *reinterpret_cast<uint4 *>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
#pragma unroll 4
    for (int k = lane * 8; k < a.K; k += 256) {
        uint4 v = make_uint4(0, 0, 0, 0), left = v;
        if (y >= 0) {
            float f[8], h[8];
            unpack(*reinterpret_cast<const uint4 *>(a.x + t * a.ldx + k), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = f[e] * r.c;
            v = pack(h);
            unpack(v, h);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fabsf(h[e]) < INFINITY ? fmaf(f[e], r.c, -h[e]) : 0.0f;
            left = pack(f);
        }
        const int64_t extent = (int64_t)a.T * a.ldxs * 2;
        __nv_bfloat16 *dst = a.xs + t * a.ldxs + k, *low = a.low + pos * a.ldxs + k;
        if (QT2_STORE_OK(dst, 16, a.xs, extent)) *reinterpret_cast<uint4 *>(dst) = v;
        if (QT2_STORE_OK(low, 16, a.low, extent)) *reinterpret_cast<uint4 *>(low) = left;
    }
}

// Two (max, sum of exp) pairs as one.
__device__ __forceinline__ float2 xent_join(const float2 &p, const float2 &q) {
    const float m = fmaxf(p.x, q.x), ref = exp_ref(m);
    return make_float2(m, p.y * __expf(p.x - ref) + q.y * __expf(q.x - ref));
}

// 32 bytes; wide: 32-byte aligned (else 16).
__device__ __forceinline__ void store_chunk(char *dst, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        st_global_v8(dst, v);
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
// A warp's 32 rows of 128 bytes, one a lane.  `dst`: the first of the four rows of the lane and its neighbours;
// `rows`: how many of these four exist.  `exchange`: chunk q of 32 bytes of all four rows goes to lane q first, so
// that a store of the warp writes 128 bytes of 8 rows and not 32 bytes of 32.  That is for tiles of at most
// kExchangeStages, which wait for their stores; in longer ones the 32 shuffles are in the way of the MMAs'
// operands (dw alone: 128 x 128 x 200000 92 us without and 68 with it, 512 x 512 x 128000 185 and 155; 1536 x 1536 x
// 100000 677 and 773).  All lanes take part.
constexpr int kExchangeStages = 8;
__device__ __forceinline__ void store_rows(uint32_t (&p)[32], char *dst, int64_t pitch, int64_t rows, bool exchange,
                                           bool wide, int lane, const void *base, int64_t extent) {
    if (!exchange) {
        dst += (lane & 3) * pitch;
        if ((lane & 3) >= rows || !QT2_STORE_OK(dst, 128, base, extent)) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t v[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) v[w] = p[j * 8 + w];
            store_chunk(dst + 32 * j, v, wide);
        }
        return;
    }
#pragma unroll
    for (int step = 1; step < 4; step *= 2) {
        const bool up = lane & step;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j & step) continue;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                uint32_t &lo = p[j * 8 + w], &hi = p[(j + step) * 8 + w];
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, step);
                if (up)
                    lo = got;
                else
                    hi = got;
            }
        }
    }
    dst += (lane & 3) * 32;
#pragma unroll
    for (int i = 0; i < 4; ++i, dst += pitch) {
        if (i >= rows || !QT2_STORE_OK(dst, 32, base, extent)) continue;
        uint32_t v[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) v[w] = p[i * 8 + w];
        store_chunk(dst, v, wide);
    }
}

// dw's rows `first` on, from a tile whose 128 columns from `col` on all exist.
__device__ __forceinline__ void dw_rows(const MmArgs &a, uint32_t (&v)[128], int64_t first, int64_t rows, int col,
                                        bool exchange, int lane, int64_t extent) {
    const int e = a.dw_f32 ? 4 : 2;
    char *dst = static_cast<char *>(a.dw) + (first * a.lddw + col) * e;
    const int64_t pitch = a.lddw * e;
    if (a.dw_f32) {
#pragma unroll
        for (int i = 0; i < 128; i += 32) {
            uint32_t p[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) p[k] = v[i + k];
            store_rows(p, dst + i * 4, pitch, rows, exchange, a.dw_wide, lane, a.dw, extent * 4);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 128; i += 64) {
        uint32_t p[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
            p[k] = *reinterpret_cast<uint32_t *>(&b2);
        }
        store_rows(p, dst + i * 2, pitch, rows, exchange, a.dw_wide, lane, a.dw, extent * 2);
    }
}

// What becomes of a tile: the thread holds columns [col, col + 128) of the tile's row `row`.
template <int MODE>
__device__ __forceinline__ void mm_epilogue(const MmArgs &a, const MmJob &b, uint32_t (&v)[128], int row, int col) {
    if (MODE == kLoss) {
        if (row >= a.T) return;
        const int valid = a.V - col;   // columns of the vocabulary from here on
        if (valid < 128) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
                if (i >= valid) v[i] = 0xFF800000u;   // -inf
        }
        float m = __uint_as_float(v[0]);
#pragma unroll
        for (int i = 1; i < 128; ++i) m = fmaxf(m, __uint_as_float(v[i]));
        const float ref = exp_ref(m);
        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
        for (int i = 0; i < 128; i += 4) {
            s0 += exp_of(__uint_as_float(v[i]) - ref);
            s1 += exp_of(__uint_as_float(v[i + 1]) - ref);
            s2 += exp_of(__uint_as_float(v[i + 2]) - ref);
            s3 += exp_of(__uint_as_float(v[i + 3]) - ref);
        }
        put(a.part, (int64_t)(col >> 7) * a.T + row, (int64_t)a.parts * a.T, make_float2(m, (s0 + s1) + (s2 + s3)));
        const int y = xent_target(a, row) - col;
        if (y >= 0 && y < 128) {
            float h = 0.0f;
#pragma unroll
            for (int i = 0; i < 128; ++i)
                if (i == y) h = __uint_as_float(v[i]);
            put(a.hit, (int64_t)row, (int64_t)a.T, h);
        }
    } else if (MODE == kProbs) {
        // rows behind the last token take part in the exchange, with no store of their own
        const int lane = row & 31, q = lane & 3, rows = a.T - row + q;
        const int y = row < a.T ? xent_target(a, row) : -1;
        const XentRow r = row < a.T ? a.rows[row] : XentRow{};
        const int at = y - (a.v0 + col), valid = a.V - (a.v0 + col);
        char *dst = reinterpret_cast<char *>(a.P) + ((int64_t)(row - q) * a.vw + col) * 2;
#pragma unroll
        for (int i = 0; i < 128; i += 64) {
            uint32_t p[32];
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                float e[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = i + k + u;
                    e[u] = exp_of(__uint_as_float(v[c]) - r.lse) * r.inv;
                    e[u] = c == at ? r.at : (y < 0 || c >= valid) ? 0.0f : e[u];
                }
                __nv_bfloat162 b2 = __floats2bfloat162_rn(e[0], e[1]);
                p[k >> 1] = *reinterpret_cast<uint32_t *>(&b2);
            }
            store_rows(p, dst + i * 2, (int64_t)a.vw * 2, rows, b.nk <= kExchangeStages, true, lane, a.P,
                       (int64_t)a.T * a.vw * 2);
        }
    } else if (!b.dw) {
        const int64_t ld = (int64_t)a.dx_n * 256;
        if (row >= a.T) return;
        float *dst = a.acc + ((int64_t)b.split * a.dx_m * 256 + row) * ld + col;
        if (!QT2_STORE_OK(dst, 512, a.acc, (int64_t)a.splits * a.dx_m * 256 * ld * 4)) return;
#pragma unroll
        for (int i = 0; i < 128; i += 8) {
            uint32_t p[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) p[k] = v[i + k];
            if (a.add) {
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const float4 o = *reinterpret_cast<const float4 *>(dst + i + k);
                    p[k] = __float_as_uint(__uint_as_float(p[k]) + o.x);
                    p[k + 1] = __float_as_uint(__uint_as_float(p[k + 1]) + o.y);
                    p[k + 2] = __float_as_uint(__uint_as_float(p[k + 2]) + o.z);
                    p[k + 3] = __float_as_uint(__uint_as_float(p[k + 3]) + o.w);
                }
            }
            st_global_v8(dst + i, p);
        }
    } else {
        const int64_t r = (int64_t)a.v0 + row;
        const int n = min(128, a.K - col);   // columns of dw from here on
        const int64_t extent = (int64_t)(a.V - 1) * a.lddw + a.K;
        if (n == 128) {
            const int lane = row & 31;
            const int64_t first = r - (lane & 3), rows = min((int64_t)a.vw - row, a.V - r) + (lane & 3);
            dw_rows(a, v, first, rows, col, b.nk <= kExchangeStages, lane, extent);
            return;
        }
        if (row >= a.vw || r >= a.V || n <= 0) return;
        if (a.dw_f32) {
            float *dst = static_cast<float *>(a.dw) + r * a.lddw + col;
            if (!QT2_STORE_OK(dst, n * 4, a.dw, extent * 4)) return;
#pragma unroll
            for (int i = 0; i < 128; i += 8) {
                if (a.dw_wide && i + 8 <= n) {
                    uint32_t p[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) p[k] = __float_as_uint(__uint_as_float(v[i + k]));
                    st_global_v8(dst + i, p);
                    continue;
                }
#pragma unroll
                for (int j = i; j < i + 8; j += 4) {
                    if (j + 4 <= n) {
                        float f[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(v[j + k]);
                        *reinterpret_cast<uint4 *>(dst + j) = pack(f);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (j + k < n) dst[j + k] = __uint_as_float(v[j + k]);
                    }
                }
            }
        } else {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dw) + r * a.lddw + col;
            if (!QT2_STORE_OK(dst, n * 2, a.dw, extent * 2)) return;
#pragma unroll
            for (int i = 0; i < 128; i += 16) {
                if (a.dw_wide && i + 16 <= n) {
                    uint32_t p[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[i + 2 * k]),
                                                                  __uint_as_float(v[i + 2 * k + 1]));
                        p[k] = *reinterpret_cast<uint32_t *>(&b2);
                    }
                    st_global_v8(dst + i, p);
                    continue;
                }
#pragma unroll
                for (int j = i; j < i + 16; j += 8) {
                    if (j + 8 <= n) {
                        float f[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v[j + k]);
                        *reinterpret_cast<uint4 *>(dst + j) = pack(f);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (j + k < n) dst[j + k] = __float2bfloat16_rn(__uint_as_float(v[j + k]));
                    }
                }
            }
        }
    }
}

// SWAP: what a token's column needs, for the epilogue's threads.
struct SwapToken {
    int y;
    XentRow row;
};
__device__ __forceinline__ SwapToken *swap_table() {
    __shared__ SwapToken tokens[kSwapN];
    return tokens;
}
template <int MODE>
__device__ __forceinline__ void swap_tokens(const MmArgs &a, int thread) {
    if (thread < kSwapN) {
        SwapToken t{-1, {}};
        if (thread < a.T) {
            t.y = xent_target(a, thread);
            if (MODE == kProbs) t.row = a.rows[thread];
        }
        swap_table()[thread] = t;
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

// The epilogue with w's rows as the tile's rows: the thread has vocabulary entry `v` of the piece, for
// 16 tokens from `first` on.  kLoss: the warp's 32 entries join the (max, sum of exp) that lane k keeps
// for token first + k.  kProbs: 32 neighbours of a row of P a store.
template <int MODE>
__device__ __forceinline__ void swap_epilogue(const MmArgs &a, int v, int first, uint32_t taddr, int lane,
                                              float2 &sum) {
    const bool in = a.v0 + v < a.V;
    uint32_t r[16];
    tmem_ld_32x32b_x16(taddr + first, r);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int t = first + k;
        if (t >= a.T) continue;
        const SwapToken token = swap_table()[t];
        const float l = in ? __uint_as_float(r[k]) : -INFINITY;
        if (MODE == kLoss) {
            float m = l;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float ref = exp_ref(m);
            float s = exp_of(l - ref);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            if (lane == k) sum = xent_join(sum, make_float2(m, s));
            if (v == token.y) put(a.hit, (int64_t)t, (int64_t)a.T, l);
        } else {
            float e = exp_of(l - token.row.lse) * token.row.inv;
            e = a.v0 + v == token.y ? token.row.at : token.y < 0 || !in ? 0.0f : e;
            __nv_bfloat16 *dst = a.P + (int64_t)t * a.vw + v;
            if (QT2_STORE_OK(dst, 2, a.P, (int64_t)a.T * a.vw * 2)) *dst = __float2bfloat16_rn(e);
        }
    }
}
// kLoss: the four lane quadrants' sums together, one pair a token and block.
__device__ __forceinline__ void swap_finish(const MmArgs &a, int ew, int lane, const float2 &sum) {
    __shared__ float2 sh[4][kSwapN];
    const int t = (ew >> 2) * 16 + lane;
    if (lane < 16) sh[ew & 3][t] = sum;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if ((ew & 3) != 0 || lane >= 16 || t >= a.T) return;
    float2 p = sh[0][t];
#pragma unroll
    for (int q = 1; q < 4; ++q) p = xent_join(p, sh[q][t]);
    put(a.part, (int64_t)blockIdx.x * a.T + t, (int64_t)a.parts * a.T, p);
}

template <int MODE, bool SWAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MmCfg<SWAP>::kThreads, 1)
    mm_pair_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmArgs a) {
    using Cfg = MmCfg<SWAP>;
    constexpr int S = Cfg::kStages;
    extern __shared__ __align__(1024) uint8_t smem_dyn[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    // barriers: full[S] empty[S] acc_full[2] acc_empty[2]
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + S * Cfg::kStageBytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 4);

    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cluster_id = blockIdx.x >> 1, num_clusters = gridDim.x >> 1;
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S);
    const uint32_t acc_full0 = smem_u32(bars + 2 * S), acc_empty0 = acc_full0 + 16;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);    // the leader's producer (expects both SMs' bytes)
            mbar_init(empty0 + 8 * s, 1);   // the MMA issuer's commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, 2 * Cfg::kEpiWarps);
        }
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

    int issued = 0;     // producer: stages whose loads were issued
    int mma_done = 0;   // MMA warp: stages whose MMAs were issued
    if (warp == 0) {
        // -------------------------------------------------------------- producer (both CTAs)
        const uint32_t full_leader0 = mapa_shared(full0, 0);
        bool ok = true;
        MmJob b;
        for (int j = 0; ok && mm_job<MODE>(a, cluster_id, num_clusters, j, b); ++j) {
            const int am = b.m * 256 + (int)rank * 128, bn = b.n * 256 + (int)rank * 128;
            const XentTile tile = mm_tile<MODE>(a, b);
            const int end = b.ks + b.nk;
            for (int ks = b.ks; ks < end + (tile.count + 63) / 64; ++ks) {
                const int it = issued, s = it % S;
                if (it >= S && !mbar_wait_warp(empty0 + 8 * s, ((it / S) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                const uint32_t st = smem_u32(base + s * Cfg::kStageBytes);
                const uint32_t fb = full_leader0 + 8 * s;
                const int k = ks * 64;
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(full0 + 8 * s, 2 * Cfg::kStageBytes);
                    if (SWAP) {
                        tma_load_2d_pair(st, &maps.w_k, k, a.v0 + bn, fb);
                        tma_load_2d_pair(st + Cfg::kA, &maps.x_k, k, (int)rank * (kSwapN / 2), fb);
                    } else if (MODE != kGrads) {
                        tma_load_2d_pair(st, &maps.x_k, k, am, fb);
                        tma_load_2d_pair(st + Cfg::kA, &maps.w_k, k, a.v0 + bn, fb);
                    } else if (!b.dw) {
                        tma_load_2d_pair(st, &maps.p_k, k, am, fb);
                        tma_load_2d_pair(st + Cfg::kA, &maps.w_mn, bn, a.v0 + k, fb);
                        tma_load_2d_pair(st + Cfg::kA + 8192, &maps.w_mn, bn + 64, a.v0 + k, fb);
                    } else if (ks >= end) {
                        const int i = (ks - end) * 64, col = (int)rank * 128;
                        tma_load_2d_pair(st, &maps.h_mn, col, tile.h + i, fb);
                        tma_load_2d_pair(st + 8192, &maps.h_mn, col + 64, tile.h + i, fb);
                        tma_load_2d_pair(st + Cfg::kA, &maps.low_mn, bn, tile.start + i, fb);
                        tma_load_2d_pair(st + Cfg::kA + 8192, &maps.low_mn, bn + 64, tile.start + i, fb);
                    } else {
                        tma_load_2d_pair(st, &maps.p_mn, am, k, fb);
                        tma_load_2d_pair(st + 8192, &maps.p_mn, am + 64, k, fb);
                        tma_load_2d_pair(st + Cfg::kA, &maps.x_mn, bn, k, fb);
                        tma_load_2d_pair(st + Cfg::kA + 8192, &maps.x_mn, bn + 64, k, fb);
                    }
                }
                __syncwarp();
                ++issued;
            }
        }
    } else if (warp == 1 && leader) {
        // -------------------------------------------------------------- MMA issuer (leader)
        // Operand tiles in shared memory, 128-byte swizzle.  K-major: 128-byte rows of 64 k, 8-row
        // groups 1 KB apart, a K = 16 step 32 bytes on.  MN-major: 64 (m or n) a 128-byte line,
        // one line a k, 8-k groups 1 KB apart, the next 64 (m or n) 8 KB on, a K = 16 step 2 KB on.
        bool ok = true;
        MmJob b;
        for (int t_iter = 0; ok && mm_job<MODE>(a, cluster_id, num_clusters, t_iter, b); ++t_iter) {
            const int buf = t_iter & 1;
            const XentTile tile = mm_tile<MODE>(a, b);
            if (t_iter >= 2 && !mbar_wait_warp(acc_empty0 + 8 * buf, ((t_iter >> 1) & 1) ^ 1)) break;
            tc_fence_after();
            const bool mn_a = MODE == kGrads && b.dw, mn_b = MODE == kGrads;
            const uint32_t idesc = Cfg::kIdesc | (mn_a ? Cfg::kIdescMnA : 0) | (mn_b ? Cfg::kIdescMnB : 0);
            const uint32_t step_a = mn_a ? 2048 : 32, step_b = mn_b ? 2048 : 32;
            const uint32_t lbo_a = mn_a ? 8192 : 16, lbo_b = mn_b ? 8192 : 16;
            for (int ks = 0; ks < b.nk + (tile.count + 63) / 64; ++ks) {
                // rows of H behind the tile's, another tile's or none, take no part
                const int steps = ks < b.nk ? 4 : min(4, (tile.count - (ks - b.nk) * 64 + kTileRows - 1) / kTileRows);
                const int it = mma_done, s = it % S;
                if (!mbar_wait_warp(full0 + 8 * s, (it / S) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(base + s * Cfg::kStageBytes);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (MODE == kGrads && kk >= steps) break;
                        tc_mma_pair_f16(tmem + 256 * buf, make_smem_desc(st + step_a * kk, lbo_a, 1024, 2),
                                        make_smem_desc(st + Cfg::kA + step_b * kk, lbo_b, 1024, 2), idesc,
                                        (ks | kk) != 0);
                    }
                    tc_commit_pair_both(empty0 + 8 * s);
                }
                __syncwarp();
                mma_done = it + 1;
            }
            if (ok) {
                if (elect_one()) tc_commit_pair_both(acc_full0 + 8 * buf);
                __syncwarp();
            }
        }
    } else if (MODE == kLoss && (warp == 2 || warp == 3)) {
        // -------------------------------------------------------------- the targets' logits, a warp a row
        for (int64_t t = (int64_t)blockIdx.x * 2 + (warp & 1); t < a.T; t += (int64_t)gridDim.x * 2) {
            const int y = xent_target(a, t);
            if (y < 0) continue;
            const float h = xent_exact(a, t, y, lane);
            if (lane == 0) put(a.exact, t, (int64_t)a.T, h);
        }
    } else if (warp >= Cfg::kEpiWarp0) {
        // -------------------------------------------------------------- epilogue (both CTAs)
        // Warp w reads TMEM lane quadrant w % 4, columns [0, 128) for warps 4..7 and [128, 256)
        // for warps 8..11; a thread holds 128 columns of one row.
        const int quad = warp & 3, ew = warp - Cfg::kEpiWarp0;
        const int cb = (ew >> 2) * 128;
        const uint32_t acc_empty_leader0 = mapa_shared(acc_empty0, 0);
        if constexpr (SWAP) swap_tokens<MODE>(a, threadIdx.x - 32 * Cfg::kEpiWarp0);
        float2 sum = make_float2(-INFINITY, 0.0f);   // SWAP, kLoss: lane k's token (ew >> 2) * 16 + k so far
        MmJob b;
        for (int t_iter = 0; mm_job<MODE>(a, cluster_id, num_clusters, t_iter, b); ++t_iter) {
            const int buf = t_iter & 1;
            if (!mbar_wait_warp(acc_full0 + 8 * buf, (t_iter >> 1) & 1)) break;
            tc_fence_after();
            if constexpr (SWAP) {
                swap_epilogue<MODE>(a, b.n * 256 + (int)rank * 128 + quad * 32 + lane, (ew >> 2) * 16,
                                    tmem + ((uint32_t)(quad * 32) << 16) + 256 * buf, lane, sum);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(acc_empty_leader0 + 8 * buf);
                continue;
            }
            const int row = b.m * 256 + (int)rank * 128 + quad * 32 + lane;
            const int col = b.n * 256 + cb;
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + 256 * buf + cb;
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 128; c += 16)
                tmem_ld_32x32b_x16(taddr + c, *reinterpret_cast<uint32_t(*)[16]>(&v[c]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(acc_empty_leader0 + 8 * buf);
            mm_epilogue<MODE>(a, b, v, row, col);
            __syncwarp();
        }
        if constexpr (SWAP && MODE == kLoss) swap_finish(a, ew, lane, sum);
    }
    // Every role ends converged.  Only after a timeout can work still be in flight: the leader
    // waits (bounded) for the loads it issued past the last consumed stage and for the last
    // issued MMAs, then both CTAs meet before TMEM is freed.
    __shared__ int consumed, issued_here;
    if (warp == 1 && leader && lane == 0) consumed = mma_done;
    if (warp == 0 && lane == 0) issued_here = issued;
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (leader && warp == 0 && lane == 0) {
        // both SMs' loads of a stage complete on the leader's barrier
        const int peer = (int)ld_shared_cluster_u32(mapa_shared(smem_u32(&issued_here), 1));
        const int last = max(issued, peer);
        for (int it = consumed; it < last; ++it) mbar_wait(full0 + 8 * (it % S), (it / S) & 1);
    }
    if (leader && warp == 1 && lane == 0 && mma_done > 0) {
        const int it = mma_done - 1;
        mbar_wait(empty0 + 8 * (it % S), (it / S) & 1);
    }
    cluster_sync_all();   // no SM frees TMEM or exits while its pair may still touch it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, Cfg::kTmemCols);
}

// loss and lse from the tiles' (max, sum) pairs: lse = M + log sum_i s_i exp(m_i - M).  A block takes
// 32 rows; its 32 warps share the pairs.  lse takes the target's exact logit h in the place of the
// tile's h' too: lse + log(1 + exp(h' - lse) (exp(h - h') - 1)).
__global__ void __launch_bounds__(1024) xent_loss_kernel(const MmArgs a, float *loss, float *lse) {
    const int parts = a.parts;
    grid_dependency();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * 32 + lane, row = blockIdx.x * 32 + warp;
    __shared__ float2 sh[32][33];
    // the row's own values, on their way while the pairs are read
    const bool live = row < a.T;
    const int in = live ? xent_target(a, row) : -1;
    const float tile = in >= 0 ? a.hit[row] : 0.0f, exact = in >= 0 ? a.exact[row] : 0.0f;
    float m = -INFINITY, s = 0.0f;
    if (t < a.T) {
        for (int i = warp; i < parts; i += 8 * 32) {
            float2 p[8];
            float n = m;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                p[k] = i + 32 * k < parts ? a.part[(int64_t)(i + 32 * k) * a.T + t] : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) n = fmaxf(n, p[k].x);
            const float ref = exp_ref(n);
            s *= __expf(m - ref);
#pragma unroll
            for (int k = 0; k < 8; ++k) s += p[k].y * __expf(p[k].x - ref);
            m = n;
        }
    }
    sh[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (!live) return;
    const float2 p = sh[lane][warp];
    float top = p.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float ref = exp_ref(top);
    float sum = p.y * __expf(p.x - ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane != 0) return;
    // the loss from differences, so that it is as exact in rows of large logits
    const float log_sum = logf(sum);
    float l = ref + log_sum, out = (ref - tile) + log_sum;
    const float off = exact - tile;
    if (in >= 0 && fabsf(off) < 16.0f) {   // not where one of them is inf or NaN
        const float more = log1pf(__expf(-out) * expm1f(off));
        l += more;
        out += more - off;
    }
    put(lse, (int64_t)row, (int64_t)a.T, l);
    put(loss, (int64_t)row, (int64_t)a.T, in >= 0 ? out : 0.0f);
    if (in < 0 && a.targets[row] != a.ignore) set_device_error(QT2_ERR_INVALID_ARG);
}

// dx = c times the sum of the splits' fp32 sums, rounded to bf16.  One thread takes 8 columns of a row.
__global__ void __launch_bounds__(256) xent_dx_kernel(const float *acc, const XentRow *row, int T, int K, int splits,
                                                      int64_t rows, int64_t ld, __nv_bfloat16 *dx, int64_t lddx) {
    grid_dependency();
    const int vecs = (K + 7) >> 3;
    const int64_t n = (int64_t)T * vecs;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / vecs;
        const int c = (int)(i - t * vecs) * 8;
        const float factor = row[t].c;
        float v[8] = {};
        for (int s = 0; s < splits; ++s) {
            const float4 *src = reinterpret_cast<const float4 *>(acc + (s * rows + t) * ld + c);
            const float4 p = src[0], q = src[1];
            v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
            v[4] += q.x; v[5] += q.y; v[6] += q.z; v[7] += q.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= factor;
        __nv_bfloat16 *dst = dx + t * lddx + c;
        const int valid = min(8, K - c);
        if (!QT2_STORE_OK(dst, valid * 2, dx, ((int64_t)(T - 1) * lddx + K) * 2)) continue;
        if (valid == 8) {
            *reinterpret_cast<uint4 *>(dst) = pack(v);
        } else {
            for (int k = 0; k < valid; ++k) dst[k] = __float2bfloat16_rn(v[k]);
        }
    }
}

}  // namespace qt2
