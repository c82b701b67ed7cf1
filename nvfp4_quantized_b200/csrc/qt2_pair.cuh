// qt2_pair.cuh -- device helpers of kernels that run on a pair of SMs (cluster of 2,
// tcgen05 cta_group::2).
#pragma once

#include "qt2_device.cuh"

namespace qt2 {

__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// The same where the barrier passes on nothing but TMEM, whose accesses tcgen05.fence::before_thread_sync
// orders: a release would also wait until this thread's earlier stores to global memory are acknowledged.
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// TMA 2D tile load into this CTA's shared memory whose completion is reported to an mbarrier
// of either CTA of the pair (cta_group::2); no multicast.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *tmap, int32_t x, int32_t y,
                                                 uint32_t bar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar_cluster)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols));
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::);
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols));
}
// Arrive once on `bar` (same offset) in both CTAs of the pair when this thread's tcgen05 work
// so far has completed.
__device__ __forceinline__ void tc_commit_pair_both(uint32_t bar) {
    const uint16_t both = 0x3;
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     bar),
                 "h"(both)
                 : "memory");
}
// Arrive on `bar` of the leader CTA only once this thread's tcgen05 work so far has completed.
__device__ __forceinline__ void tc_commit_pair_leader(uint32_t bar) {
    const uint16_t leader_only = 0x1;
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     bar),
                 "h"(leader_only)
                 : "memory");
}

// 32-byte global store (sm_100 256-bit vector store); the address is 32-byte aligned.
__device__ __forceinline__ void st_global_v8(void *dst, const uint32_t (&p)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(p[0]), "r"(p[1]), "r"(p[2]),
                 "r"(p[3]), "r"(p[4]), "r"(p[5]), "r"(p[6]), "r"(p[7])
                 : "memory");
}

}  // namespace qt2
