// qt2_train.cu -- the training operators' library: kernel launchers and the C ABI declared in
// include/qt2_train.h (layer norm, the head's softmax cross entropy, the gated feed-forward product,
// the norm of queries and keys with the rotation, gradient norm and clipping, AdamW).
//
// One translation unit, with a device status word, fault hook and caches of its own.  Built for
// sm_100a only into libqt2_train.so.
#include <cmath>

#include "qt2_internal.h"
#include "qt2_train.h"
#include "qt2_host.cuh"
#include "qt2_device.cuh"
#include "norm_kernels.cuh"
#include "grad_kernels.cuh"
#include "xent_kernels.cuh"
#include "gated_kernels.cuh"
#include "rope_kernels.cuh"
#include "adamw_kernels.cuh"

using namespace qt2;

namespace {

cudaStream_t as_stream(qt2_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool dim_ok(int64_t d) { return d > 0 && d < (int64_t(1) << 30); }
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int d) { return d == QT2_DTYPE_BF16 || d == QT2_DTYPE_F32; }
bool ld_shape_ok(int64_t ld, int64_t cols) { return ld >= cols && ld < (int64_t(1) << 40); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

qt2_status check_workspace(const void *ws, size_t have, size_t need) {
    if (!ws || have < need) return QT2_ERR_WORKSPACE;
    return aligned(ws, kWsAlign) ? QT2_OK : QT2_ERR_ALIGN;
}

// Every kernel is launched so that its start overlaps the end of the one before it in the stream
// (grid_dependency).
template <class T>
struct Same {
    using type = T;
};
template <class... P>
cudaError_t launch_cluster(void (*kernel)(P...), int cluster, dim3 grid, int threads, size_t smem, cudaStream_t s,
                           const typename Same<P>::type &...args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = cluster ? 2 : 1;   // 0: the kernel's own cluster, or none
    void *list[] = {const_cast<void *>(static_cast<const void *>(&args))...};
    return cudaLaunchKernelExC(&c, reinterpret_cast<const void *>(kernel), list);
}
template <class... P>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                   const typename Same<P>::type &...args) {
    return launch_cluster(kernel, 0, grid, threads, smem, s, args...);
}

// Blocks of a launch that is one cluster, for n shares of work.
int cluster_blocks(int64_t n) { return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : 8; }

// ------------------------------------------------------------------------------- layer norm
// Resident blocks of a kernel on this device, asked once a device.
template <class F>
cudaError_t resident_blocks(PerDeviceOnce &once, std::atomic<int> *blocks, F kernel, int threads, int smem,
                            int64_t *n) {
    const cudaError_t e = once.run([&] {
        int v = 0;
        const cudaError_t f = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kernel, threads, smem);
        if (f == cudaSuccess) blocks[current_device()].store(std::max(1, v) * sm_count());
        return f;
    });
    if (e == cudaSuccess) *n = blocks[current_device()].load();
    return e;
}
template <class T, int V, int B>
cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    static PerDeviceOnce attr, once;
    static std::atomic<int> blocks[kMaxDevices];
    // weights and biases as fp32, and B rows a warp
    auto smem = [](int warps) { return 32 * V * 16 * (8 / (int)sizeof(T) + B * warps); };
    int64_t n = 0;
    cudaError_t e = attr.run([&] {
        return cudaFuncSetAttribute(layernorm_fwd_kernel<T, V, B>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    smem(8));
    });
    if (e == cudaSuccess) e = resident_blocks(once, blocks, layernorm_fwd_kernel<T, V, B>, 256, smem(8), &n);
    if (e != cudaSuccess) return e;
    // fewer rows than the SMs have warps: spread over more SMs, fewer warps of a block have some
    const int64_t steps = ceil_div(a.rows, B);
    NormArgs b = a;
    b.warps = (int)std::min<int64_t>(8, ceil_div(steps, sm_count()));
    return launch(layernorm_fwd_kernel<T, V, B>, (unsigned)std::min(n, ceil_div(steps, b.warps)), 256, smem(b.warps),
                  s, b);
}
template <class T, int G>
cudaError_t launch_norm_fwd_short(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    constexpr int B = 4;
    static PerDeviceOnce once;
    static std::atomic<int> blocks[kMaxDevices];
    int64_t n = 0;
    const cudaError_t e = resident_blocks(once, blocks, layernorm_fwd_short_kernel<T, G, B>, 256, 0, &n);
    if (e != cudaSuccess) return e;
    return launch(layernorm_fwd_short_kernel<T, G, B>, (unsigned)std::min(n, ceil_div(a.rows, 256 / G * B)), 256, 0, s,
                  a);
}
template <class T, int G, bool HOLD>
cudaError_t launch_norm_fwd_group(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    constexpr int V = (HOLD ? 16 : 32) / kVec<T>, kGroups = 1024 / G, kMost = 222 * 1024;
    constexpr int kWeights = HOLD ? 0 : 2 * 32 * G * (int)sizeof(float);
    static_assert(kWeights + kGroups * G * V * 16 <= kMost, "a row a group");
    static PerDeviceOnce once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(layernorm_fwd_group_kernel<T, G, V, HOLD>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    });
    if (e != cudaSuccess) return e;
    NormArgs b = a;
    const int rows = kGroups * norm_row_bytes<T>(a.cols);
    b.slots = std::min(3, (kMost - kWeights) / rows);
    return launch(layernorm_fwd_group_kernel<T, G, V, HOLD>,
                  (unsigned)std::min<int64_t>(sm_count(), ceil_div(a.rows, kGroups)), 1024,
                  kWeights + b.slots * rows, s, b);
}
template <class T>
cudaError_t launch_norm_fwd_long(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(layernorm_fwd_long_kernel<T>, (unsigned)a.rows, kNormThreads, 0, s, a);
}
template <class T>
cudaError_t norm_fwd(const NormArgs &a, cudaStream_t s) {
    const int64_t n = ceil_div(a.cols, kVec<T>);   // 16-byte vectors a row
    if (n <= 4) return launch_norm_fwd_short<T, 4>(a, s);
    if (n <= 8) return launch_norm_fwd_short<T, 8>(a, s);
    if (n <= 16) return launch_norm_fwd_short<T, 16>(a, s);
    if (n <= 32) return launch_norm_fwd<T, 1, 4>(a, s);
    if (n <= 64) return launch_norm_fwd<T, 2, 4>(a, s);
    if (n <= 128) return launch_norm_fwd<T, 4, 2>(a, s);
    if (n <= 256) return launch_norm_fwd<T, 8, 1>(a, s);
    if (n <= 512) return launch_norm_fwd<T, 16, 1>(a, s);
    // bf16: 32 columns a thread, so that two groups more share an SM's barriers (8192 x 8192: 50 us, with 16
    // columns and the weights in registers 68); fp32 has the bytes to cover them (16384 x 4096: 88 us, 93 with 32)
    if constexpr (sizeof(T) == 2) {
        if (a.cols <= 8192) return launch_norm_fwd_group<T, 256, false>(a, s);
    } else {
        if (a.cols <= 4096) return launch_norm_fwd_group<T, 256, true>(a, s);
        if (a.cols <= 8192) return launch_norm_fwd_group<T, 512, true>(a, s);
    }
    if (a.cols <= 16384) return launch_norm_fwd_group<T, 1024, true>(a, s);
    return launch_norm_fwd_long<T>(a, s);
}

// The backward pass's threads a row (0: the row is too long for registers), rows a block and step,
// and its blocks: resident ones, since every block leaves a partial
// sum of dw and db, and no more of them than it takes for every one to run as many steps (rows too
// long: the slices of the rows that dw and db are summed in).
// Rows of at most one step of eight blocks: one cluster of blocks, which add up dw and db themselves
// (1 x 2048 bf16: 7.9 us, two launches 10.0; with two steps, 128 x 2048, 10.7 and 10.0).
struct NormBwdPlan {
    int threads, step, blocks, cluster;
};
template <class T>
NormBwdPlan norm_bwd_plan(int64_t rows, int64_t cols) {
    auto ring = [](auto r) {
        using R = decltype(r);
        return NormBwdPlan{32, R::kGroups * R::B, 148, 0};
    };
    NormBwdPlan p = cols <= 64      ? NormBwdPlan{8, 64, 148 * 2, 0}
                    : cols <= 256   ? ring(NormRing<T, 32, 8>{})
                    : cols <= 512   ? ring(NormRing<T, 32, 16>{})
                    : cols <= 1024  ? ring(NormRing<T, 64, 16>{})
                    : cols <= 2048  ? ring(NormRing<T, 128, 16>{})
                    : cols <= 4096  ? ring(NormRing<T, 256, 16>{})
                    : cols <= 8192  ? ring(NormRing<T, 512, 16>{})
                    : cols <= 16384 ? ring(NormRing<T, 512, 32>{})
                                    : NormBwdPlan{0, 16, 64, 0};
    const int64_t steps = ceil_div(rows, p.step);
    p.blocks = (int)ceil_div(steps, ceil_div(steps, p.blocks));
    p.cluster = 0;
    if (p.threads == 32 && steps <= 8) {
        p.cluster = cluster_blocks(steps);
        p.blocks = p.cluster;
    }
    return p;
}

template <class T, int G, int V, int B>
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(layernorm_bwd_kernel<T, G, V, B>, (unsigned)a.splits, 256, 0, s, a);
}
template <class T, int G, int C, bool WHOLE>
cudaError_t launch_norm_bwd_ring(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    using R = NormRing<T, G, C>;
    static PerDeviceOnce once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(layernorm_bwd_ring_kernel<T, G, C, WHOLE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, R::bytes(R::kColumns));
    });
    if (e != cudaSuccess) return e;
    return launch_cluster(layernorm_bwd_ring_kernel<T, G, C, WHOLE>, a.cluster, (unsigned)a.splits, R::kGroups * G,
                          R::bytes(a.cols), s, a);
}
template <class T, int G, int C>
cudaError_t norm_bwd_ring(const NormArgs &a, cudaStream_t s) {
    return a.cols % kVec<T> ? launch_norm_bwd_ring<T, G, C, false>(a, s)
                            : launch_norm_bwd_ring<T, G, C, true>(a, s);
}
cudaError_t launch_norm_dw(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(layernorm_dw_kernel, dim3((unsigned)ceil_div(a.cols, 32), 2), 1024, 0, s, a);
}
template <class T>
cudaError_t launch_norm_dx_long(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(layernorm_dx_long_kernel<T>, (unsigned)a.rows, kNormThreads, 0, s, a);
}
template <class T>
cudaError_t launch_norm_dw_long(const NormArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    const dim3 grid((unsigned)ceil_div(a.cols, kNormThreads * kVec<T>), (unsigned)a.splits);
    return launch(layernorm_dw_long_kernel<T>, grid, kNormThreads, 0, s, a);
}
template <class T>
cudaError_t norm_bwd(const NormArgs &a, int threads, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (threads == 0) {   // the sums before dx, which may be dy
        if (a.part) e = launch_norm_dw_long<T>(a, s);
        if (e == cudaSuccess && a.y) e = launch_norm_dx_long<T>(a, s);
    } else {
        e = a.cols <= 64     ? launch_norm_bwd<T, 8, 8 / kVec<T>, 2>(a, s)
            : a.cols <= 256  ? norm_bwd_ring<T, 32, 8>(a, s)
            : a.cols <= 512  ? norm_bwd_ring<T, 32, 16>(a, s)
            : a.cols <= 1024 ? norm_bwd_ring<T, 64, 16>(a, s)
            : a.cols <= 2048 ? norm_bwd_ring<T, 128, 16>(a, s)
            : a.cols <= 4096 ? norm_bwd_ring<T, 256, 16>(a, s)
            : a.cols <= 8192 ? norm_bwd_ring<T, 512, 16>(a, s)
                             : norm_bwd_ring<T, 512, 32>(a, s);
    }
    if (e == cudaSuccess && a.part && !a.cluster) e = launch_norm_dw(a, s);
    return e;
}

// ------------------------------------------------------------------------------- head loss
// The plan depends on the sizes alone, so that the workspace queries need no device: 74 pairs.
constexpr int kPairs = 74;
// Of P.  8192 tokens, hidden 4096, vocabulary 128000, backward: pieces of 64 MB 20.3 ms, 256 MB 19.3 ms,
// 512 MB 19.0 ms, 1 GB 18.8 ms (fewer passes over the sums of dx, fewer uneven ends of launches).
constexpr int64_t kPieceBytes = 512 << 20;
// Of x, what a group of the tokens' tiles shares while the vocabulary goes by: it has to stay in L2 (8192
// tokens, hidden 4096: x in one group of 64 MB 5.68 ms, in two of 32 MB 5.44 ms, in four 5.84 ms, forward).
constexpr int64_t kGroupBytes = 32 << 20;
constexpr int kJobStages = 4;                // what a tile's start and end cost, in stages of K = 64
// A tile of dw takes its stages and those of the tokens that have their target in it, or as long as its 128 KB (bf16)
// take to leave: 2.2 us in all, eight stages' time.
int64_t dw_job(int64_t T, int64_t num_v) {
    return std::max<int64_t>(ceil_div(T, 64) + ceil_div(T, 64 * num_v), 4) + kJobStages;
}

struct XentPlan {
    int64_t num_m, num_v, num_k;   // 256-wide tiles of T, V and K
    bool swap;                     // the tiles of logits have w's rows as their rows
    int parts;                     // (max, sum) pairs a row of logits
    int64_t piece;                 // vocabulary entries of a piece, a multiple of 256
    int pieces, splits;
};

XentPlan xent_plan(int64_t T, int64_t K, int64_t V) {
    XentPlan p;
    p.num_m = ceil_div(T, 256);
    p.num_v = ceil_div(V, 256);
    p.num_k = ceil_div(K, 256);
    p.swap = T < kSwapN;
    p.parts = p.swap ? 2 * (int)std::min<int64_t>(p.num_v, kPairs) : 2 * (int)p.num_v;
    const int64_t most = std::max<int64_t>(1, kPieceBytes / (512 * T));
    p.pieces = (int)ceil_div(p.num_v, most);
    p.piece = ceil_div(p.num_v, p.pieces) * 256;
    p.pieces = (int)ceil_div(p.num_v * 256, p.piece);
    // dx's jobs are cut along the vocabulary where that shortens the launch: the pairs' even share
    // of its stages or the longest pair's dx jobs, and what the sums that each cut adds cost to write and read.
    // An eighth of those jobs besides: while they run on some of the pairs, these read w no faster than their MMAs
    // take it, and what comes after them is levelled by estimate (16 tokens, hidden 4096, vocabulary 64000: two cuts
    // 338 us, four 299, nine 301).
    const int64_t nks = p.piece / 64, dx = p.num_m * p.num_k;
    const int64_t dw = p.piece / 256 * p.num_k * dw_job(T, p.num_v);
    double best = 0;
    for (int s = 1; s <= 16 && s * 16 <= std::max<int64_t>(16, nks); ++s) {
        const int64_t job = ceil_div(nks, s) + kJobStages;
        const double share = (double)(dx * s * job + dw) / kPairs, longest = (double)(ceil_div(dx * s, kPairs) * job);
        const double cost = std::max(share, longest) + longest / 8 + (double)dx * s * std::min<int64_t>(T, 256) / 1024;
        if (s == 1 || cost < best) {
            best = cost;
            p.splits = s;
        }
    }
    return p;
}

struct XentFwdWs {
    float2 *part;
    float *hit, *exact;
    size_t bytes;
};
XentFwdWs xent_fwd_ws(const XentPlan &p, int64_t T, void *ws) {
    Carve c(ws);
    XentFwdWs w;
    w.part = reinterpret_cast<float2 *>(c.take((size_t)p.parts * T * sizeof(float2)));
    w.hit = reinterpret_cast<float *>(c.take((size_t)T * sizeof(float)));
    w.exact = reinterpret_cast<float *>(c.take((size_t)T * sizeof(float)));
    w.bytes = c.used;
    return w;
}
struct XentBwdWs {
    __nv_bfloat16 *P, *xs, *low;
    __nv_bfloat16 *H;
    int64_t h_rows;
    int *count, *pos;
    XentTile *tile;
    XentRow *rows;
    float *acc;
    size_t bytes;
};
XentBwdWs xent_bwd_ws(const XentPlan &p, int64_t T, int64_t K, void *ws) {
    Carve c(ws);
    XentBwdWs w;
    w.P = reinterpret_cast<__nv_bfloat16 *>(c.take((size_t)T * p.piece * 2));
    w.xs = reinterpret_cast<__nv_bfloat16 *>(c.take((size_t)T * ceil_div(K, 64) * 128));
    w.low = reinterpret_cast<__nv_bfloat16 *>(c.take((size_t)T * ceil_div(K, 64) * 128));
    w.h_rows = T + (kTileRows - 1) * std::min<int64_t>(p.num_v, T);   // no more tiles have targets
    w.H = reinterpret_cast<__nv_bfloat16 *>(c.take((size_t)w.h_rows * 512));
    w.count = reinterpret_cast<int *>(c.take((size_t)(p.num_v + 1) * ceil_div(T, kSortTokens) * sizeof(int)));
    w.pos = reinterpret_cast<int *>(c.take((size_t)T * sizeof(int)));
    w.tile = reinterpret_cast<XentTile *>(c.take((size_t)p.num_v * sizeof(XentTile)));
    w.rows = reinterpret_cast<XentRow *>(c.take((size_t)T * sizeof(XentRow)));
    w.acc = reinterpret_cast<float *>(c.take((size_t)p.splits * p.num_m * p.num_k * 65536 * sizeof(float)));
    w.bytes = c.used;
    return w;
}

bool encode_bf16(CUtensorMap *m, const void *p, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
    return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, (uint64_t)cols, (uint64_t)rows, (uint64_t)ld * 2, 64,
                          (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE, bool SWAP>
cudaError_t launch_mm(const MmMaps &maps, const MmArgs &a, int64_t jobs, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    static PerDeviceOnce once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(mm_pair_kernel<MODE, SWAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    MmCfg<SWAP>::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    const int64_t clusters = std::min<int64_t>(jobs, kPairs);
    return launch(mm_pair_kernel<MODE, SWAP>, (unsigned)(2 * clusters), MmCfg<SWAP>::kThreads,
                  MmCfg<SWAP>::kSmemBytes, s, maps, a);
}

cudaError_t launch_xent_loss(const MmArgs &a, float *loss, float *lse, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(xent_loss_kernel, (unsigned)ceil_div(a.T, 32), 1024, 0, s, a, loss, lse);
}

cudaError_t launch_xent_rows(const MmArgs &a, const float *lse, const float *dloss, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(xent_rows_kernel, (unsigned)ceil_div(a.T, 8), 256, 0, s, a, lse, dloss);
}

cudaError_t launch_xent_sort(const MmArgs &a, int blocks, int phases, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(xent_sort_kernel, (unsigned)blocks, 1024, 0, s, a, phases);
}
cudaError_t xent_sort(const MmArgs &a, cudaStream_t s) {
    if (a.words == 1) return launch_xent_sort(a, 1, kCount | kScan | kRank, s);
    cudaError_t e = launch_xent_sort(a, a.words, kCount, s);
    if (e == cudaSuccess) e = launch_xent_sort(a, 1, kScan, s);
    return e == cudaSuccess ? launch_xent_sort(a, a.words, kRank, s) : e;
}

cudaError_t launch_xent_dx(const MmArgs &a, void *dx, int64_t lddx, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    const int64_t n = (int64_t)a.T * ceil_div(a.K, 8);
    const int64_t blocks = std::min<int64_t>(ceil_div(n, 256), (int64_t)sm_count() * 16);
    return launch(xent_dx_kernel, (unsigned)blocks, 256, 0, s, a.acc, a.rows, a.T, a.K, a.splits,
                  (int64_t)a.dx_m * 256, (int64_t)a.dx_n * 256, static_cast<__nv_bfloat16 *>(dx), lddx);
}

// T, K and V, and x's and w's elements (which bound the workspaces' sizes) below 2^44.
bool xent_dims_ok(int64_t T, int64_t K, int64_t V) {
    return dim_ok(T) && dim_ok(K) && dim_ok(V) && T * K < (int64_t(1) << 44) && V * K < (int64_t(1) << 44);
}

qt2_status xent_check(const void *x, const void *w, const int64_t *targets, int64_t T, int64_t K, int64_t V,
                      int64_t ldx, int64_t ldw) {
    if (!x || !w || !targets) return QT2_ERR_INVALID_ARG;
    if (!xent_dims_ok(T, K, V) || !ld_shape_ok(ldx, K) || !ld_shape_ok(ldw, K)) return QT2_ERR_SHAPE;
    if (std::max(ldx, ldw) >= (int64_t(1) << 39)) return QT2_ERR_SHAPE;   // a tensor map's rows: below 2^40 bytes
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(targets, 8) || ldx % 8 || ldw % 8) return QT2_ERR_ALIGN;
    return QT2_OK;
}

// ------------------------------------------------------------------------------- gated product
bool views_given(const qt2_nvfp4_view *v) { return v && v->codes && v->scales && v->tensor_scale; }
bool view_aligned(const qt2_nvfp4_view *v) {
    return aligned(v->codes, 16) && aligned(v->scales, 16) && aligned(v->tensor_scale, 4);
}

// Multiples of 128, and no more than 2^31 steps of a tile in all.
bool gated_dims_ok(int64_t M, int64_t F, int64_t K) {
    const int64_t most = int64_t(1) << 44;
    if (!dim_ok(M) || !dim_ok(F) || !dim_ok(K) || M % 128 || F % 128 || K % 128) return false;
    if (M * F >= most || M * K >= most || F * K >= most) return false;
    return ceil_div(M, 256) * (F / 128) <= INT32_MAX / ceil_div(K, 256);
}

// Codes in boxes of 128 rows, scale atoms as rows of K/64 512-byte atoms, `atoms` rows a box.
bool encode_view(CUtensorMap *codes, CUtensorMap *scales, const qt2_nvfp4_view *v, int64_t R, int64_t K, int atoms) {
    return encode_tmap_2d(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, v->codes, (uint64_t)K / 2, (uint64_t)R,
                          (uint64_t)K / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode_tmap_2d(scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, v->scales, (uint64_t)K, (uint64_t)R / 128,
                          (uint64_t)K * 8, 256, (uint32_t)atoms, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <bool BWD, int ACT>
cudaError_t launch_gated(const GatedMaps &maps, const GatedArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    using Cfg = GatedCfg<BWD>;
    static PerDeviceOnce once;
    const cudaError_t e = once.run([] {
        // the backward kernel's warps wait for registers that the launch has to have
        cudaFuncAttributes f;
        if (const cudaError_t q = cudaFuncGetAttributes(&f, gated_pair_kernel<BWD, ACT>)) return q;
        if (BWD && f.numRegs < Cfg::kRegs) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(gated_pair_kernel<BWD, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Cfg::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    const int64_t tiles = ceil_div(a.M, 256) * ceil_div(a.F, BWD ? 256 : 128);
    const int64_t clusters = std::max<int64_t>(1, std::min<int64_t>(tiles, sm_count() / 2));
    return launch(gated_pair_kernel<BWD, ACT>, (unsigned)(2 * clusters), Cfg::kThreads, Cfg::kSmemBytes, s,
                  maps, a);
}
template <bool BWD>
cudaError_t gated(const GatedMaps &maps, const GatedArgs &a, int act, cudaStream_t s) {
    return act == QT2_ACT_SILU ? launch_gated<BWD, QT2_ACT_SILU>(maps, a, s)
                               : launch_gated<BWD, QT2_ACT_GELU_TANH>(maps, a, s);
}

// ------------------------------------------------------------------------------- queries and keys
// Heads that a group of lanes takes at a time.  Forward, 32768 x 16+16 x 128 bf16: 1 head 168 us, 2 heads 125, 4
// heads 108, 8 heads, which spill, 140; backward 1 head 282, 2 heads 196, 4 heads 163, 8 heads 171.
template <class T, int N>
constexpr int kQkRows = std::max(1, (sizeof(T) == 2 ? 4 : 2) / N);

// Blocks of the backward pass: each leaves a share of dw.
int64_t qk_bwd_blocks(int64_t T, int64_t Hq, int64_t Hk) {
    return std::min<int64_t>(148 * 2, ceil_div(T * (Hq + Hk), kQkThreads / 32));
}

template <class T, int G, int N, bool PAIRS>
cudaError_t launch_qk_fwd(const QkArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    constexpr int U = kQkRows<T, N>, kGroups = 32 / G;
    const int64_t warps = ceil_div(a.T * ceil_div(a.heads[0], U), kGroups) + ceil_div(a.T * ceil_div(a.heads[1], U), kGroups);
    return launch(qk_norm_rope_fwd_kernel<T, G, N, U, PAIRS>, (unsigned)ceil_div(warps, kQkThreads / 32), kQkThreads, 0,
                  s, a);
}
template <class T, int G, int N, bool PAIRS>
cudaError_t launch_qk_bwd(const QkArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(qk_norm_rope_bwd_kernel<T, G, N, kQkRows<T, N>, PAIRS>, (unsigned)a.parts, kQkThreads,
                  a.D * (kQkThreads / 32) * sizeof(float), s, a);
}
template <bool BWD, class T, int G, int N>
cudaError_t qk_launch(const QkArgs &a, bool pairs, cudaStream_t s) {
    if constexpr (BWD)
        return pairs ? launch_qk_bwd<T, G, N, true>(a, s) : launch_qk_bwd<T, G, N, false>(a, s);
    else
        return pairs ? launch_qk_fwd<T, G, N, true>(a, s) : launch_qk_fwd<T, G, N, false>(a, s);
}
template <bool BWD, class T>
cudaError_t qk_norm_rope(const QkArgs &a, int pairing, cudaStream_t s) {
    const int slots = a.D / 8;
    const bool pairs = pairing == QT2_ROPE_PAIRS;
    if (slots <= 8) return qk_launch<BWD, T, 8, 1>(a, pairs, s);
    if (slots <= 16) return qk_launch<BWD, T, 16, 1>(a, pairs, s);
    if (slots <= 32) return qk_launch<BWD, T, 32, 1>(a, pairs, s);
    if (slots <= 64) return qk_launch<BWD, T, 32, 2>(a, pairs, s);
    return qk_launch<BWD, T, 32, 4>(a, pairs, s);
}
cudaError_t launch_qk_dw(const QkArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(qk_dw_kernel, dim3((unsigned)ceil_div(a.D, 32), 2), 1024, 0, s, a);
}

bool qk_dims_ok(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    const int64_t heads = int64_t(1) << 20;
    return dim_ok(T) && Hq >= 0 && Hk >= 0 && Hq < heads && Hk < heads && Hq + Hk > 0 &&
           T * (Hq + Hk) < (int64_t(1) << 32) && D > 0 && D <= 1024 && D % 8 == 0;
}
// T tokens of H heads of D elements, one inside the other either way, none over another.
bool qk_strides_ok(int64_t T, int64_t H, int64_t D, int64_t ld, int64_t hs) {
    const int64_t most = int64_t(1) << 32;
    if (ld < 0 || hs < 0 || ld >= most || hs >= most) return false;
    const __int128 heads = (__int128)(H - 1) * hs + D, tokens = (__int128)(T - 1) * ld + D;   // of a token, of a head
    return ((H == 1 || hs >= D) && (T == 1 || ld >= heads)) || ((T == 1 || ld >= D) && (H == 1 || hs >= tokens));
}
qt2_status qk_check(const void *x, int x_dtype, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t ldx, int64_t hsx,
                    const void *wq, const void *wk, int w_dtype, float eps, const int64_t *positions, const float *cos,
                    const float *sin, int64_t P, int64_t R, int pairing) {
    if (!x || !dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !(eps >= 0.0f) || std::isinf(eps) ||
        (pairing != QT2_ROPE_HALVES && pairing != QT2_ROPE_PAIRS) || (R != 0 && (!cos || !sin)))
        return QT2_ERR_INVALID_ARG;
    if (!qk_dims_ok(T, Hq, Hk, D) || R < 0 || R > D || R % 8 || !qk_strides_ok(T, Hq + Hk, D, ldx, hsx))
        return QT2_ERR_SHAPE;
    if (R != 0 && (!dim_ok(P) || (!positions && T > P))) return QT2_ERR_SHAPE;
    if (!aligned(x, 16) || ldx % 8 || hsx % 8 || !aligned(wq, 16) || !aligned(wk, 16) || !aligned(positions, 8) ||
        !aligned(cos, 16) || !aligned(sin, 16))
        return QT2_ERR_ALIGN;
    return QT2_OK;
}
QkArgs qk_args(const void *x, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t ldx, int64_t hsx, const void *wq,
               const void *wk, int w_dtype, float eps, const int64_t *positions, const float *cos, const float *sin,
               int64_t P, int64_t R) {
    QkArgs a{};
    a.x = x;
    a.w[0] = wq;
    a.w[1] = wk;
    a.pos = positions;
    a.cos = cos;
    a.sin = sin;
    a.P = P;
    a.T = T;
    a.heads[0] = (int)Hq;
    a.heads[1] = (int)Hk;
    a.D = (int)D;
    a.R = (int)R;
    a.ldx = (uint32_t)ldx;
    a.hsx = (uint32_t)hsx;
    a.w_f32 = w_dtype == QT2_DTYPE_F32;
    a.eps = eps;
    return a;
}

// ------------------------------------------------------------------------------- gradients
qt2_status grad_check(const qt2_grad *g, int64_t count, bool with_out) {
    if (!g) return QT2_ERR_INVALID_ARG;
    if (count <= 0 || count > (int64_t(1) << 30)) return QT2_ERR_SHAPE;
    for (int64_t i = 0; i < count; ++i) {
        if (!dtype_ok(g[i].dtype)) return QT2_ERR_INVALID_ARG;
        if (g[i].numel < 0 || g[i].numel >= (int64_t(1) << 42)) return QT2_ERR_SHAPE;
        if (g[i].numel == 0) continue;
        if (!g[i].grad || (with_out && !g[i].out)) return QT2_ERR_INVALID_ARG;
        const uintptr_t e = g[i].dtype == QT2_DTYPE_F32 ? 4 : 2;
        if (!aligned(g[i].grad, e) || (with_out && !aligned(g[i].out, e))) return QT2_ERR_ALIGN;
    }
    return QT2_OK;
}

// Launches beyond one a full table that tensors of many TB add.
int64_t grad_over(const qt2_grad *g, int64_t count) {
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) chunks += ceil_div(g[i].numel, 4 * kGradChunk) + 1;
    return chunks / (INT32_MAX / 2);
}
// The next launch's tensors: fills t from g[at...], skipping empty ones; returns the next `at`.
template <int N>
int64_t grad_table(GradTable<N> &t, const qt2_grad *g, int64_t at, int64_t count) {
    t.count = 0;
    std::memset(t.f32, 0, sizeof t.f32);
    t.first[0] = 0;
    for (; at < count && t.count < N; ++at) {
        if (g[at].numel == 0) continue;
        const int k = t.count, esz = g[at].dtype == QT2_DTYPE_F32 ? 4 : 2;
        const int64_t bytes = (int64_t)(reinterpret_cast<uintptr_t>(g[at].grad) & 15) + g[at].numel * esz;
        const int64_t next = t.first[k] + ceil_div(bytes, 16 * kGradChunk);
        if (next > INT32_MAX) break;   // 64 TB a launch
        ++t.count;
        t.grad[k] = g[at].grad;
        t.out[k] = g[at].out;
        t.numel[k] = g[at].numel;
        t.first[k + 1] = (int32_t)next;
        if (esz == 4) t.f32[k >> 5] |= 1u << (k & 31);
    }
    return at;
}
// A block takes about four chunks: short enough shares that the SMs finish together, whatever
// the tensors' sizes, long enough that looking the tensor up does not show.  Of the norm's launch at most
// kGradBlocks, which leave a partial sum each.
constexpr int kGradBlocks = 148 * 32;
template <int N>
int grad_blocks(const GradTable<N> &t, int most) {
    const int chunks = t.first[t.count];
    return std::min(std::min(chunks, most), std::max(148 * 4, chunks / 4));
}
// Up to so many chunks the launch is one cluster of as many blocks, which forms the norm itself (40 chunks on
// eight blocks: 16.3 us for norm and clipping, with a launch for the end 12.5).
constexpr int kGradAlone = 8;

template <int N>
cudaError_t launch_grad_norm(const GradTable<N> &t, double *part, float *norm, int blocks, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch_cluster(grad_norm_kernel<N>, norm ? blocks : 0, blocks, kGradThreads, 0, s, t, part, norm);
}
cudaError_t launch_grad_norm_end(const double *part, int n, float *norm, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(grad_norm_end_kernel, 1, kGradThreads, 0, s, part, n, norm);
}
template <int N>
cudaError_t launch_grad_clip(const GradTable<N> &t, const float *norm, float max_norm, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    return launch(grad_clip_kernel<N>, grad_blocks(t, INT32_MAX), kGradThreads, 0, s, t, norm, max_norm);
}

template <int N>
cudaError_t grad_norm(const qt2_grad *grads, int64_t count, float *norm, double *part, cudaStream_t s) {
    GradTable<N> t;
    int n = 0;
    for (int64_t at = 0; at < count;) {
        at = grad_table(t, grads, at, count);
        if (t.count == 0) break;
        const bool alone = n == 0 && at == count && t.first[t.count] <= kGradAlone;
        const int blocks = alone ? cluster_blocks(t.first[t.count]) : grad_blocks(t, kGradBlocks);
        const cudaError_t e = launch_grad_norm(t, part + n, alone ? norm : nullptr, blocks, s);
        if (e != cudaSuccess || alone) return e;
        n += blocks;
    }
    return launch_grad_norm_end(part, n, norm, s);
}
template <int N>
cudaError_t grad_clip(const qt2_grad *grads, int64_t count, const float *norm, float max_norm, cudaStream_t s) {
    GradTable<N> t;
    for (int64_t at = 0; at < count;) {
        at = grad_table(t, grads, at, count);
        if (t.count == 0) break;
        const cudaError_t e = launch_grad_clip(t, norm, max_norm, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// ------------------------------------------------------------------------------- AdamW
qt2_status adamw_check(const qt2_adamw_tensor *t, int64_t count) {
    if (!t) return QT2_ERR_INVALID_ARG;
    if (count <= 0 || count > (int64_t(1) << 30)) return QT2_ERR_SHAPE;
    for (int64_t i = 0; i < count; ++i) {
        const qt2_adamw_tensor &a = t[i];
        const bool e4m3 = a.state == QT2_STATE_E4M3;
        if (!dtype_ok(a.param_dtype) || !dtype_ok(a.grad_dtype) || (a.state != QT2_STATE_F32 && !e4m3) ||
            !std::isfinite(a.weight_decay) || (a.master && a.param_dtype == QT2_DTYPE_F32))
            return QT2_ERR_INVALID_ARG;
        if (a.numel < 0 || a.numel >= (int64_t(1) << 40)) return QT2_ERR_SHAPE;
        if (a.numel == 0) continue;
        if (!a.param || !a.grad || !a.m || !a.v || (e4m3 && (!a.m_scale || !a.v_scale))) return QT2_ERR_INVALID_ARG;
        const uintptr_t p = a.param_dtype == QT2_DTYPE_F32 ? 4 : 2, g = a.grad_dtype == QT2_DTYPE_F32 ? 4 : 2;
        const uintptr_t s = e4m3 ? 1 : 4;
        if (!aligned(a.param, p) || !aligned(a.grad, g) || !aligned(a.m, s) || !aligned(a.v, s) || !aligned(a.master, 4) ||
            (e4m3 && (!aligned(a.m_scale, 4) || !aligned(a.v_scale, 4))))
            return QT2_ERR_ALIGN;
    }
    return QT2_OK;
}

// Elements by which a tensor's arrays all start behind a multiple of four; -1 where they differ, or where
// blocks of 256, which count from the first element, would not be made of whole vectors.
int adamw_head(const qt2_adamw_tensor &a) {
    auto behind = [](const void *p, int size) { return (int)(reinterpret_cast<uintptr_t>(p) / size & 3); };
    const bool e4m3 = a.state == QT2_STATE_E4M3;
    const int s = e4m3 ? 1 : 4, head = behind(a.grad, a.grad_dtype == QT2_DTYPE_F32 ? 4 : 2);
    const bool same = behind(a.param, a.param_dtype == QT2_DTYPE_F32 ? 4 : 2) == head && behind(a.m, s) == head &&
                      behind(a.v, s) == head && (!a.master || behind(a.master, 4) == head);
    return same && (!e4m3 || head == 0) ? head : -1;
}

// The types that a kernel is compiled for, as a number below 12.
int adamw_kind(const qt2_adamw_tensor &a) {
    const int param = a.master ? kAdamMaster : a.param_dtype == QT2_DTYPE_F32 ? kAdamF32 : kAdamBf16;
    return param * 4 + (a.grad_dtype == QT2_DTYPE_F32 ? 2 : 0) + (a.state == QT2_STATE_E4M3 ? 1 : 0);
}

// The next launch's tensors, those of one kind from tensors[at] on; returns the next `at`.
template <int N>
int64_t adamw_table(AdamTable<N> &t, const qt2_adamw_tensor *tensors, int64_t at, int64_t count, int kind) {
    t.count = 0;
    t.first[0] = 0;
    for (; at < count && t.count < N; ++at) {
        const qt2_adamw_tensor &a = tensors[at];
        if (a.numel == 0 || adamw_kind(a) != kind) continue;
        const int k = t.count, head = adamw_head(a);
        const int64_t next = t.first[k] + ceil_div(std::max(0, head) + a.numel, kAdamChunk);
        if (next > INT32_MAX / 2) break;   // a launch's chunks, and the blocks' next ones
        ++t.count;
        t.param[k] = a.param;
        t.master[k] = a.master;
        t.grad[k] = a.grad;
        t.m[k] = a.m;
        t.v[k] = a.v;
        t.m_scale[k] = a.m_scale;
        t.v_scale[k] = a.v_scale;
        t.numel[k] = a.numel;
        t.first[k + 1] = (int32_t)next;
        t.id[k] = (int32_t)at;
        t.decay[k] = a.weight_decay;
        t.flags[k] = (uint8_t)((head >= 0 ? kAdamVectors : 0) + std::max(0, head) * kAdamHead);
    }
    return at;
}

template <int N, bool E4M3, AdamParam P, bool GF32>
cudaError_t launch_adamw(const AdamTable<N> &t, const AdamArgs &a, cudaStream_t s) {
    QT2_LAUNCH_SITE();
    static PerDeviceOnce once;
    static std::atomic<int> blocks[kMaxDevices];
    int64_t n = 0;
    const auto kernel = adamw_kernel<N, E4M3, P, GF32>;
    const cudaError_t e = resident_blocks(once, blocks, kernel, kAdamThreads, 0, &n);
    if (e != cudaSuccess) return e;
    return launch(kernel, (unsigned)std::min<int64_t>(n, t.first[t.count]), kAdamThreads, 0, s, t, a);
}
template <int N, AdamParam P>
cudaError_t launch_adamw(const AdamTable<N> &t, int kind, const AdamArgs &a, cudaStream_t s) {
    return (kind & 3) == 0   ? launch_adamw<N, false, P, false>(t, a, s)
           : (kind & 3) == 1 ? launch_adamw<N, true, P, false>(t, a, s)
           : (kind & 3) == 2 ? launch_adamw<N, false, P, true>(t, a, s)
                             : launch_adamw<N, true, P, true>(t, a, s);
}
template <int N>
cudaError_t adamw(const qt2_adamw_tensor *tensors, int64_t count, const AdamArgs &a, cudaStream_t s) {
    uint32_t kinds = 0;
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].numel) kinds |= 1u << adamw_kind(tensors[i]);
    AdamTable<N> t;
    for (int kind = 0; kind < 12; ++kind) {
        if (!(kinds >> kind & 1)) continue;
        for (int64_t at = 0; at < count;) {
            at = adamw_table(t, tensors, at, count, kind);
            if (t.count == 0) break;
            const cudaError_t e = kind / 4 == kAdamBf16  ? launch_adamw<N, kAdamBf16>(t, kind, a, s)
                                  : kind / 4 == kAdamF32 ? launch_adamw<N, kAdamF32>(t, kind, a, s)
                                                         : launch_adamw<N, kAdamMaster>(t, kind, a, s);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

extern "C" {

qt2_status qt2_train_device_status(qt2_stream_t stream, int *code) {
    QT2_TRACE();
    if (!code) return QT2_ERR_INVALID_ARG;
    if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return QT2_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int)) != cudaSuccess) return QT2_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess) return QT2_ERR_CUDA;
    *code = v;
    return QT2_OK;
}

void qt2_train_set_fault_hook(qt2_fault_hook hook, void *user) {
    g_fault_user.store(user, std::memory_order_release);
    g_fault_hook.store(hook, std::memory_order_release);
}

int qt2_train_build_checked(void) {
#ifdef QT2_CHECKED
    return 1;
#else
    return 0;
#endif
}

qt2_status qt2_layernorm_fwd(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *weight,
                             const void *bias, int w_dtype, float eps, void *y, int64_t ldy, float *mean, float *rstd,
                             qt2_stream_t stream) {
    QT2_TRACE();
    if (!x || !y || !dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !(eps >= 0.0f) || std::isinf(eps))
        return QT2_ERR_INVALID_ARG;
    if (!dim_ok(rows) || !dim_ok(cols) || !ld_shape_ok(ldx, cols) || !ld_shape_ok(ldy, cols)) return QT2_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(y, 16) || ldx % 8 || ldy % 8 || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return QT2_ERR_ALIGN;
    if (const qt2_status st = check_device()) return st;
    NormArgs a{};
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.cols = (int)cols;
    a.ldx = ldx;
    a.ldy = ldy;
    a.w_f32 = w_dtype == QT2_DTYPE_F32;
    a.eps = eps;
    const cudaStream_t s = as_stream(stream);
    return from_cuda(x_dtype == QT2_DTYPE_F32 ? norm_fwd<float>(a, s) : norm_fwd<__nv_bfloat16>(a, s));
}

qt2_status qt2_layernorm_bwd_workspace_size(int64_t rows, int64_t cols, size_t *bytes) {
    if (!bytes) return QT2_ERR_INVALID_ARG;
    if (!dim_ok(rows) || !dim_ok(cols)) return QT2_ERR_SHAPE;
    const int blocks = std::max(norm_bwd_plan<float>(rows, cols).blocks,
                                norm_bwd_plan<__nv_bfloat16>(rows, cols).blocks);
    *bytes = align_up((size_t)blocks * 2 * cols * sizeof(float), kWsAlign);
    return QT2_OK;
}

qt2_status qt2_layernorm_bwd(const void *dy, int64_t lddy, const void *x, int x_dtype, int64_t rows, int64_t cols,
                             int64_t ldx, const void *weight, int w_dtype, const float *mean, const float *rstd,
                             void *dx, int64_t lddx, void *dweight, void *dbias, void *workspace, size_t ws_bytes,
                             qt2_stream_t stream) {
    QT2_TRACE();
    if (!dy || !x || !mean || !rstd || (!dx && !dweight && !dbias) || !dtype_ok(x_dtype) || !dtype_ok(w_dtype))
        return QT2_ERR_INVALID_ARG;
    if (!dim_ok(rows) || !dim_ok(cols) || !ld_shape_ok(ldx, cols) || !ld_shape_ok(lddy, cols) ||
        (dx && !ld_shape_ok(lddx, cols)))
        return QT2_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(dy, 16) || ldx % 8 || lddy % 8 || (dx && (!aligned(dx, 16) || lddx % 8)) ||
        !aligned(weight, 16) || !aligned(dweight, 16) || !aligned(dbias, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
        return QT2_ERR_ALIGN;
    size_t need = 0;
    if (const qt2_status st = qt2_layernorm_bwd_workspace_size(rows, cols, &need)) return st;
    if (const qt2_status st = check_workspace(workspace, ws_bytes, need)) return st;
    if (const qt2_status st = check_device()) return st;
    NormArgs a{};
    a.x = x;
    a.dy = dy;
    a.w = weight;
    a.y = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.rows = rows;
    a.cols = (int)cols;
    a.ldx = ldx;
    a.lddy = lddy;
    a.ldy = lddx;
    a.w_f32 = w_dtype == QT2_DTYPE_F32;
    a.part = dweight || dbias ? static_cast<float *>(workspace) : nullptr;
    const NormBwdPlan p = x_dtype == QT2_DTYPE_F32 ? norm_bwd_plan<float>(rows, cols)
                                                   : norm_bwd_plan<__nv_bfloat16>(rows, cols);
    a.splits = p.blocks;
    a.cluster = p.cluster;
    a.dw = dweight;
    a.db = dbias;
    const cudaStream_t s = as_stream(stream);
    return from_cuda(x_dtype == QT2_DTYPE_F32 ? norm_bwd<float>(a, p.threads, s)
                                              : norm_bwd<__nv_bfloat16>(a, p.threads, s));
}

qt2_status qt2_linear_xent_fwd_workspace_size(int64_t T, int64_t K, int64_t V, size_t *bytes) {
    if (!bytes) return QT2_ERR_INVALID_ARG;
    if (!xent_dims_ok(T, K, V)) return QT2_ERR_SHAPE;
    *bytes = xent_fwd_ws(xent_plan(T, K, V), T, nullptr).bytes;
    return QT2_OK;
}

qt2_status qt2_linear_xent_fwd(const void *x, const void *w, const int64_t *targets, int64_t T, int64_t K, int64_t V,
                               int64_t ldx, int64_t ldw, int64_t ignore_index, float *loss, float *lse,
                               void *workspace, size_t ws_bytes, qt2_stream_t stream) {
    QT2_TRACE();
    if (!loss || !lse) return QT2_ERR_INVALID_ARG;
    if (const qt2_status st = xent_check(x, w, targets, T, K, V, ldx, ldw)) return st;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return QT2_ERR_ALIGN;
    const XentPlan p = xent_plan(T, K, V);
    if (const qt2_status st = check_workspace(workspace, ws_bytes, xent_fwd_ws(p, T, nullptr).bytes)) return st;
    if (const qt2_status st = check_device()) return st;
    const XentFwdWs ws = xent_fwd_ws(p, T, workspace);
    MmMaps maps{};
    if (!encode_bf16(&maps.x_k, x, K, T, ldx, p.swap ? kSwapN / 2 : 128) ||
        !encode_bf16(&maps.w_k, w, K, V, ldw, 128))
        return QT2_ERR_CUDA;
    MmArgs a{};
    a.T = (int)T;
    a.K = (int)K;
    a.V = (int)V;
    a.vw = (int)(p.num_v * 256);
    a.targets = targets;
    a.ignore = ignore_index;
    a.part = ws.part;
    a.parts = p.parts;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.w = static_cast<const __nv_bfloat16 *>(w);
    a.ldx = ldx;
    a.ldw = ldw;
    a.hit = ws.hit;
    a.exact = ws.exact;
    a.num_m = (int)p.num_m;
    a.group_m = (int)std::min<int64_t>(p.num_m, std::max<int64_t>(8, kGroupBytes / (512 * K)));
    a.num_n = (int)p.num_v;
    const cudaStream_t s = as_stream(stream);
    cudaError_t e = p.swap ? launch_mm<kLoss, true>(maps, a, p.num_v, s)
                             : launch_mm<kLoss, false>(maps, a, p.num_m * p.num_v, s);
    if (e == cudaSuccess) e = launch_xent_loss(a, loss, lse, s);
    return from_cuda(e);
}

qt2_status qt2_linear_xent_bwd_workspace_size(int64_t T, int64_t K, int64_t V, size_t *bytes) {
    if (!bytes) return QT2_ERR_INVALID_ARG;
    if (!xent_dims_ok(T, K, V)) return QT2_ERR_SHAPE;
    *bytes = xent_bwd_ws(xent_plan(T, K, V), T, K, nullptr).bytes;
    return QT2_OK;
}

qt2_status qt2_linear_xent_bwd(const void *x, const void *w, const int64_t *targets, const float *lse,
                               const float *dloss, int64_t T, int64_t K, int64_t V, int64_t ldx, int64_t ldw,
                               int64_t ignore_index, void *dx, int64_t lddx, void *dw, int dw_dtype, int64_t lddw,
                               void *workspace, size_t ws_bytes, qt2_stream_t stream) {
    QT2_TRACE();
    if (!lse || !dloss || (!dx && !dw) || (dw && !dtype_ok(dw_dtype))) return QT2_ERR_INVALID_ARG;
    if (const qt2_status st = xent_check(x, w, targets, T, K, V, ldx, ldw)) return st;
    if ((dx && !ld_shape_ok(lddx, K)) || (dw && !ld_shape_ok(lddw, K))) return QT2_ERR_SHAPE;
    if (!aligned(lse, 4) || !aligned(dloss, 4) || (dx && (!aligned(dx, 16) || lddx % 8)) ||
        (dw && (!aligned(dw, 16) || lddw % 8)))
        return QT2_ERR_ALIGN;
    const XentPlan p = xent_plan(T, K, V);
    if (const qt2_status st = check_workspace(workspace, ws_bytes, xent_bwd_ws(p, T, K, nullptr).bytes)) return st;
    if (const qt2_status st = check_device()) return st;
    const XentBwdWs ws = xent_bwd_ws(p, T, K, workspace);
    MmMaps maps{};
    if (!encode_bf16(&maps.x_k, x, K, T, ldx, p.swap ? kSwapN / 2 : 128) ||
        !encode_bf16(&maps.w_k, w, K, V, ldw, 128) || !encode_bf16(&maps.x_mn, ws.xs, K, T, ceil_div(K, 64) * 64, 64) ||
        !encode_bf16(&maps.low_mn, ws.low, K, T, ceil_div(K, 64) * 64, 64) ||
        !encode_bf16(&maps.h_mn, ws.H, 256, ws.h_rows, 256, 64) ||
        !encode_bf16(&maps.w_mn, w, K, V, ldw, 64))
        return QT2_ERR_CUDA;
    MmArgs a{};
    a.T = (int)T;
    a.K = (int)K;
    a.V = (int)V;
    a.targets = targets;
    a.ignore = ignore_index;
    a.P = ws.P;
    a.num_m = (int)p.num_m;
    a.group_m = (int)std::min<int64_t>(p.num_m, std::max<int64_t>(8, kGroupBytes / (512 * K)));
    a.splits = p.splits;
    a.dx_m = (int)p.num_m;
    a.dx_n = (int)p.num_k;
    a.acc = ws.acc;
    a.rows = ws.rows;
    a.xs = dw ? ws.xs : nullptr;
    a.low = ws.low;
    a.H = ws.H;
    a.h_rows = ws.h_rows;
    a.count = ws.count;
    a.words = (int)ceil_div(T, kSortTokens);
    a.pos = ws.pos;
    a.tile = ws.tile;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.ldx = ldx;
    a.ldxs = ceil_div(K, 64) * 64;
    a.w = static_cast<const __nv_bfloat16 *>(w);
    a.ldw = ldw;
    a.dw = dw;
    a.lddw = lddw;
    a.dw_f32 = dw_dtype == QT2_DTYPE_F32;
    a.dw_wide = aligned(dw, 32) && lddw * (a.dw_f32 ? 4 : 2) % 32 == 0;
    const cudaStream_t s = as_stream(stream);
    cudaError_t e = dw ? xent_sort(a, s) : cudaSuccess;
    if (e == cudaSuccess) e = launch_xent_rows(a, lse, dloss, s);
    if (e != cudaSuccess) return from_cuda(e);
    for (int i = 0; i < p.pieces; ++i) {
        a.v0 = (int)(i * p.piece);
        a.vw = (int)std::min<int64_t>(p.piece, p.num_v * 256 - a.v0);
        a.num_n = a.vw / 256;
        a.add = i > 0;
        a.splits = (int)std::min<int64_t>(p.splits, a.vw / 64);
        a.dx_jobs = dx ? a.splits * a.dx_m * a.dx_n : 0;
        a.dw_jobs = dw ? a.num_n * (int)p.num_k : 0;
        a.lead = (int)((a.vw / 64 / a.splits + kJobStages) / dw_job(T, p.num_v));
        if (!encode_bf16(&maps.p_k, ws.P, a.vw, T, a.vw, 128) || !encode_bf16(&maps.p_mn, ws.P, a.vw, T, a.vw, 64))
            return QT2_ERR_CUDA;
        e = p.swap ? launch_mm<kProbs, true>(maps, a, a.num_n, s)
                   : launch_mm<kProbs, false>(maps, a, (int64_t)a.num_m * a.num_n, s);
        if (e == cudaSuccess) e = launch_mm<kGrads, false>(maps, a, (int64_t)a.dx_jobs + a.dw_jobs, s);
        if (e != cudaSuccess) return from_cuda(e);
    }
    if (!dx) return QT2_OK;
    a.splits = p.splits;
    return from_cuda(launch_xent_dx(a, dx, lddx, s));
}

qt2_status qt2_gemm_nvfp4_gated(const qt2_nvfp4_view *a, const qt2_nvfp4_view *b_gate, const qt2_nvfp4_view *b_up,
                                int64_t M, int64_t F, int64_t K, float alpha, int act, void *gate, void *up,
                                int64_t ldgu, void *h, int64_t ldh, qt2_stream_t stream) {
    QT2_TRACE();
    if (!views_given(a) || !views_given(b_gate) || !views_given(b_up) || !h || !gate != !up ||
        (act != QT2_ACT_SILU && act != QT2_ACT_GELU_TANH))
        return QT2_ERR_INVALID_ARG;
    if (!gated_dims_ok(M, F, K) || !ld_shape_ok(ldh, F) || (gate && !ld_shape_ok(ldgu, F))) return QT2_ERR_SHAPE;
    if (!view_aligned(a) || !view_aligned(b_gate) || !view_aligned(b_up) || !aligned(h, 16) || ldh % 8 ||
        (gate && (!aligned(gate, 16) || !aligned(up, 16) || ldgu % 8)))
        return QT2_ERR_ALIGN;
    if (const qt2_status st = check_device()) return st;
    GatedMaps maps{};
    if (!encode_view(&maps.a, &maps.sfa, a, M, K, 1) || !encode_view(&maps.b[0], &maps.sfb[0], b_gate, F, K, 1) ||
        !encode_view(&maps.b[1], &maps.sfb[1], b_up, F, K, 1))
        return QT2_ERR_CUDA;
    GatedArgs g{};
    g.ga = a->tensor_scale;
    g.gb[0] = b_gate->tensor_scale;
    g.gb[1] = b_up->tensor_scale;
    g.alpha = alpha;
    g.M = (int)M;
    g.F = (int)F;
    g.K = (int)K;
    // all of x's rows at a time where x is the smaller operand, so that the weights stream once (16384 x 4096 x 14336: 16
    // rows 997 us, all 980; one row 1126); else F first (32768 x 2048 x 5632: one row 453 us, 16 rows 468).  The rule does
    // not look at K: at 16384 x 8192 x 28672 x's 75 MB do not stay in L2 beside the outputs, and 16 rows take 3406 us
    // where all take 3950 (one row 4574)
    g.group_m = M < 2 * F ? (int)ceil_div(M, 256) : 1;
    g.gate = static_cast<__nv_bfloat16 *>(gate);
    g.up = static_cast<__nv_bfloat16 *>(up);
    g.ldgu = ldgu;
    g.h = static_cast<__nv_bfloat16 *>(h);
    g.ldh = ldh;
    return from_cuda(gated<false>(maps, g, act, as_stream(stream)));
}

qt2_status qt2_gemm_nvfp4_gated_bwd(const qt2_nvfp4_view *a, const qt2_nvfp4_view *b, int64_t M, int64_t F, int64_t K,
                                    float alpha, int act, const void *gate, const void *up, int64_t ldgu, void *dgate,
                                    void *dup, int64_t lddgu, void *h, int64_t ldh, qt2_stream_t stream) {
    QT2_TRACE();
    if (!views_given(a) || !views_given(b) || !gate || !up || !dgate || !dup ||
        (act != QT2_ACT_SILU && act != QT2_ACT_GELU_TANH))
        return QT2_ERR_INVALID_ARG;
    if (!gated_dims_ok(M, F, K) || !ld_shape_ok(ldgu, F) || !ld_shape_ok(lddgu, F) || (h && !ld_shape_ok(ldh, F)))
        return QT2_ERR_SHAPE;
    if (ldgu >= (int64_t(1) << 39)) return QT2_ERR_SHAPE;   // a tensor map's rows: below 2^40 bytes
    if (!view_aligned(a) || !view_aligned(b) || !aligned(gate, 16) || !aligned(up, 16) || ldgu % 8 ||
        !aligned(dgate, 16) || !aligned(dup, 16) || lddgu % 8 || (h && (!aligned(h, 16) || ldh % 8)))
        return QT2_ERR_ALIGN;
    if (const qt2_status st = check_device()) return st;
    GatedMaps maps{};
    // gate and up in boxes of 32 rows x 64 columns
    auto encode_piece = [&](CUtensorMap *m, const void *p) {
        return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, (uint64_t)F, (uint64_t)M, (uint64_t)ldgu * 2, 64, 32,
                              CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!encode_view(&maps.a, &maps.sfa, a, M, K, 1) || !encode_view(&maps.b[0], &maps.sfb[0], b, F, K, 2) ||
        !encode_piece(&maps.gate, gate) || !encode_piece(&maps.up, up))
        return QT2_ERR_CUDA;
    GatedArgs g{};
    g.ga = a->tensor_scale;
    g.gb[0] = b->tensor_scale;
    g.alpha = alpha;
    g.M = (int)M;
    g.F = (int)F;
    g.K = (int)K;
    // 8 rows of tiles: what the streams of gate, up and outputs push out of L2 is soon used again (16384 x 4096 x 14336:
    // 1 row 816 us, 4 787, 8 771, 16 772, 32 791; 32768 x 2048 x 5632: 482 to 490 all)
    g.group_m = 8;
    g.gate = static_cast<__nv_bfloat16 *>(const_cast<void *>(gate));
    g.up = static_cast<__nv_bfloat16 *>(const_cast<void *>(up));
    g.ldgu = ldgu;
    g.dgate = static_cast<__nv_bfloat16 *>(dgate);
    g.dup = static_cast<__nv_bfloat16 *>(dup);
    g.lddgu = lddgu;
    g.h = static_cast<__nv_bfloat16 *>(h);
    g.ldh = ldh;
    return from_cuda(gated<true>(maps, g, act, as_stream(stream)));
}

qt2_status qt2_qk_norm_rope_fwd(const void *x, int x_dtype, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t ldx,
                                int64_t hsx, const void *wq, const void *wk, int w_dtype, float eps,
                                const int64_t *positions, const float *cos, const float *sin, int64_t P, int64_t R,
                                int pairing, void *y, int64_t ldy, int64_t hsy, qt2_stream_t stream) {
    QT2_TRACE();
    if (!y) return QT2_ERR_INVALID_ARG;
    if (const qt2_status st = qk_check(x, x_dtype, T, Hq, Hk, D, ldx, hsx, wq, wk, w_dtype, eps, positions, cos, sin, P,
                                       R, pairing))
        return st;
    if (!qk_strides_ok(T, Hq + Hk, D, ldy, hsy)) return QT2_ERR_SHAPE;
    if (!aligned(y, 16) || ldy % 8 || hsy % 8) return QT2_ERR_ALIGN;
    if (const qt2_status st = check_device()) return st;
    QkArgs a = qk_args(x, T, Hq, Hk, D, ldx, hsx, wq, wk, w_dtype, eps, positions, cos, sin, P, R);
    a.y = y;
    a.ldy = (uint32_t)ldy;
    a.hsy = (uint32_t)hsy;
    const cudaStream_t s = as_stream(stream);
    return from_cuda(x_dtype == QT2_DTYPE_F32 ? qk_norm_rope<false, float>(a, pairing, s)
                                              : qk_norm_rope<false, __nv_bfloat16>(a, pairing, s));
}

qt2_status qt2_qk_norm_rope_bwd_workspace_size(int64_t T, int64_t Hq, int64_t Hk, int64_t D, size_t *bytes) {
    if (!bytes) return QT2_ERR_INVALID_ARG;
    if (!qk_dims_ok(T, Hq, Hk, D)) return QT2_ERR_SHAPE;
    *bytes = align_up((size_t)qk_bwd_blocks(T, Hq, Hk) * 2 * D * sizeof(float), kWsAlign);
    return QT2_OK;
}

qt2_status qt2_qk_norm_rope_bwd(const void *dy, int64_t lddy, int64_t hsdy, const void *x, int x_dtype, int64_t T,
                                int64_t Hq, int64_t Hk, int64_t D, int64_t ldx, int64_t hsx, const void *wq,
                                const void *wk, int w_dtype, float eps, const int64_t *positions, const float *cos,
                                const float *sin, int64_t P, int64_t R, int pairing, void *dx, int64_t lddx,
                                int64_t hsdx, void *dwq, void *dwk, void *workspace, size_t ws_bytes,
                                qt2_stream_t stream) {
    QT2_TRACE();
    if (!dy || (!dx && !dwq && !dwk)) return QT2_ERR_INVALID_ARG;
    if (const qt2_status st = qk_check(x, x_dtype, T, Hq, Hk, D, ldx, hsx, wq, wk, w_dtype, eps, positions, cos, sin, P,
                                       R, pairing))
        return st;
    if (!qk_strides_ok(T, Hq + Hk, D, lddy, hsdy) || (dx && !qk_strides_ok(T, Hq + Hk, D, lddx, hsdx)))
        return QT2_ERR_SHAPE;
    if (!aligned(dy, 16) || lddy % 8 || hsdy % 8 || (dx && (!aligned(dx, 16) || lddx % 8 || hsdx % 8)) ||
        !aligned(dwq, 16) || !aligned(dwk, 16))
        return QT2_ERR_ALIGN;
    size_t need = 0;
    if (const qt2_status st = qt2_qk_norm_rope_bwd_workspace_size(T, Hq, Hk, D, &need)) return st;
    if (const qt2_status st = check_workspace(workspace, ws_bytes, need)) return st;
    if (const qt2_status st = check_device()) return st;
    QkArgs a = qk_args(x, T, Hq, Hk, D, ldx, hsx, wq, wk, w_dtype, eps, positions, cos, sin, P, R);
    a.dy = dy;
    a.lddy = (uint32_t)lddy;
    a.hsdy = (uint32_t)hsdy;
    a.y = dx;
    a.ldy = (uint32_t)lddx;
    a.hsy = (uint32_t)hsdx;
    a.dw[0] = dwq;
    a.dw[1] = dwk;
    a.part = dwq || dwk ? static_cast<float *>(workspace) : nullptr;
    a.parts = (int)qk_bwd_blocks(T, Hq, Hk);
    const cudaStream_t s = as_stream(stream);
    cudaError_t e = x_dtype == QT2_DTYPE_F32 ? qk_norm_rope<true, float>(a, pairing, s)
                                             : qk_norm_rope<true, __nv_bfloat16>(a, pairing, s);
    if (e == cudaSuccess && a.part) e = launch_qk_dw(a, s);
    return from_cuda(e);
}

qt2_status qt2_grad_norm_workspace_size(const qt2_grad *grads, int64_t count, size_t *bytes) {
    if (!bytes) return QT2_ERR_INVALID_ARG;
    if (const qt2_status st = grad_check(grads, count, false)) return st;
    *bytes = (size_t)(ceil_div(count, kGradLarge) + grad_over(grads, count)) *
             kGradBlocks * sizeof(double);
    return QT2_OK;
}

qt2_status qt2_grad_norm(const qt2_grad *grads, int64_t count, float *norm, void *workspace, size_t ws_bytes,
                         qt2_stream_t stream) {
    QT2_TRACE();
    if (!norm) return QT2_ERR_INVALID_ARG;
    size_t need = 0;
    if (const qt2_status st = qt2_grad_norm_workspace_size(grads, count, &need)) return st;
    if (!aligned(norm, 4)) return QT2_ERR_ALIGN;
    if (const qt2_status st = check_workspace(workspace, ws_bytes, need)) return st;
    if (const qt2_status st = check_device()) return st;
    double *part = static_cast<double *>(workspace);
    const cudaStream_t s = as_stream(stream);
    return from_cuda(count <= kGradSmall    ? grad_norm<kGradSmall>(grads, count, norm, part, s)
                     : count <= kGradMiddle ? grad_norm<kGradMiddle>(grads, count, norm, part, s)
                                            : grad_norm<kGradLarge>(grads, count, norm, part, s));
}

qt2_status qt2_grad_clip(const qt2_grad *grads, int64_t count, const float *norm, float max_norm,
                         qt2_stream_t stream) {
    QT2_TRACE();
    if (!norm || !(max_norm >= 0.0f)) return QT2_ERR_INVALID_ARG;
    if (const qt2_status st = grad_check(grads, count, true)) return st;
    if (!aligned(norm, 4)) return QT2_ERR_ALIGN;
    if (const qt2_status st = check_device()) return st;
    const cudaStream_t s = as_stream(stream);
    return from_cuda(count <= kGradSmall    ? grad_clip<kGradSmall>(grads, count, norm, max_norm, s)
                     : count <= kGradMiddle ? grad_clip<kGradMiddle>(grads, count, norm, max_norm, s)
                                            : grad_clip<kGradLarge>(grads, count, norm, max_norm, s));
}

qt2_status qt2_adamw(const qt2_adamw_tensor *tensors, int64_t count, const float *lr, const int64_t *step, double beta1,
                     double beta2, float eps, const float *norm, float max_norm, uint64_t seed, qt2_stream_t stream) {
    QT2_TRACE();
    if (!lr || !step || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0f) ||
        std::isinf(eps) || (norm && !(max_norm >= 0.0f)))
        return QT2_ERR_INVALID_ARG;
    if (const qt2_status st = adamw_check(tensors, count)) return st;
    if (!aligned(lr, 4) || !aligned(step, 8) || !aligned(norm, 4)) return QT2_ERR_ALIGN;
    if (const qt2_status st = check_device()) return st;
    AdamArgs a{};
    a.lr = lr;
    a.norm = norm;
    a.step = step;
    a.log_b1 = std::log(beta1);
    a.log_b2 = std::log(beta2);
    a.b1 = (float)beta1;
    a.b2 = (float)beta2;
    a.one_b1 = (float)(1.0 - beta1);
    a.one_b2 = (float)(1.0 - beta2);
    a.unit = eps > 0.0f && eps < 0x1p-126f ? 0x1p24f : 1.0f;
    a.eps = eps * a.unit;
    a.max_norm = max_norm;
    a.minus_zero = -0.0f;
    for (uint32_t r = 0; r < 10; ++r) {
        a.key0[r] = (uint32_t)seed + r * kPhiloxKey0;
        a.key1[r] = (uint32_t)(seed >> 32) + r * kPhiloxKey1;
    }
    const cudaStream_t s = as_stream(stream);
    return from_cuda(count <= kAdamSmall ? adamw<kAdamSmall>(tensors, count, a, s)
                                         : adamw<kAdamLarge>(tensors, count, a, s));
}

}  // extern "C"
