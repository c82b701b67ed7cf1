// qt2_host.cuh -- host code shared by the libraries: fault injection, per-device caches, TMA
// descriptors, the device check and the workspace carver.  Each library includes it in one
// translation unit and has its own hook and caches.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "qt2_internal.h"

namespace qt2 {

// ---------------------------------------------------------------------------------------------
// host-side fault injection and per-device caches
// ---------------------------------------------------------------------------------------------
static std::atomic<qt2_fault_hook> g_fault_hook{nullptr};
static std::atomic<void *> g_fault_user{nullptr};

int fault_at(const char *site) {
    const qt2_fault_hook h = g_fault_hook.load(std::memory_order_acquire);
    if (h == nullptr) return kFaultNone;
    const int a = h(site, g_fault_user.load(std::memory_order_acquire));
    return (a == kFaultFail || a == kFaultSkip) ? a : kFaultNone;
}

int current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return dev;
}

// One-time set-up per device (function attributes, occupancy): f() runs with the device
// current until it has succeeded once there.  A process that drives several GPUs sets every
// kernel up on each of them.
struct PerDeviceOnce {
    std::atomic<int> done[kMaxDevices];
    template <class F>
    cudaError_t run(F &&f) {
        const int dev = current_device();
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
        const cudaError_t e = f();
        if (e == cudaSuccess) done[dev].store(1, std::memory_order_release);
        return e;
    }
};

// Launch sites consult the fault hook: a failure is reported as a failed launch, a skip as a
// successful one, and in both cases nothing is launched.
#define QT2_LAUNCH_SITE()                                        \
    do {                                                         \
        const int fa_ = fault_at("launch");                      \
        if (fa_ == kFaultFail) return cudaErrorLaunchFailure;    \
        if (fa_ == kFaultSkip) return cudaSuccess;               \
    } while (0)

static cudaError_t memset_async(void *p, size_t n, cudaStream_t s) {
    const int fa = fault_at("memset");
    if (fa == kFaultFail) return cudaErrorInvalidValue;
    if (fa == kFaultSkip) return cudaSuccess;
    return cudaMemsetAsync(p, 0, n, s);
}

static int sm_count() {
    static std::atomic<int> cached[kMaxDevices];
    const int dev = current_device();
    if (dev < 0 || dev >= kMaxDevices) return 148;
    int v = cached[dev].load();
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) {
            cudaGetLastError();
            v = 148;
        }
        cached[dev].store(v);
    }
    return v;
}

// ---------------------------------------------------------------------------------------------
// TMA descriptors (driver entry point fetched through the runtime; no libcuda link needed)
// ---------------------------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

bool encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t outer,
                    uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz) {
    const int fa = fault_at("tensor_map");
    if (fa == kFaultFail) return false;
    if (fa == kFaultSkip) {
        std::memset(map, 0, sizeof(*map));
        return true;
    }
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {row_stride_bytes};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, dtype, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// ---------------------------------------------------------------------------------------------
// checks and workspaces
// ---------------------------------------------------------------------------------------------
static constexpr size_t kWsAlign = 256;

static size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static qt2_status check_device() {
    const int fa = fault_at("device");
    if (fa == kFaultFail) return QT2_ERR_DEVICE;
    if (fa == kFaultSkip) return QT2_OK;
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
        cudaGetLastError();
        return QT2_ERR_DEVICE;
    }
    if (dev < 64) {
        int v = cached[dev].load();
        if (v == 1) return QT2_OK;
        if (v == 2) return QT2_ERR_DEVICE;
    }
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
        cudaGetLastError();
        return QT2_ERR_DEVICE;
    }
    const bool ok = (major == 10 && minor == 0);
    if (dev < 64) cached[dev].store(ok ? 1 : 2);
    return ok ? QT2_OK : QT2_ERR_DEVICE;
}

static qt2_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return QT2_OK;
    cudaGetLastError();   // reported here, not by the caller's next CUDA call
    return QT2_ERR_CUDA;
}

// Bump allocator over the caller's workspace.
struct Carve {
    uint8_t *base;
    size_t used = 0;
    explicit Carve(void *b) : base(static_cast<uint8_t *>(b)) {}
    uint8_t *take(size_t bytes) {
        uint8_t *p = base ? base + used : nullptr;
        used = align_up(used + bytes, kWsAlign);
        return p;
    }
};

}  // namespace qt2
