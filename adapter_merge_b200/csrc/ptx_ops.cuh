// Inline-PTX wrappers of the operators between the adapted linears, beside
// ptx.cuh: waits of a whole warp, thread-block clusters and CTA pairs.  Every
// spin-wait here is bounded by kWaitLimitNs too.
#pragma once

#include "ptx.cuh"

namespace af {

// As mbar_wait, for waits that come every few hundred cycles: the clock and
// the abort flag are looked at only after a run of tries.
__device__ __forceinline__ bool mbar_wait_hot(uint64_t* bar, uint32_t parity, volatile int* abort)
{
    uint64_t t0 = 0;
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        const uint64_t now = globaltimer_ns();
        if (!t0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
}

// The same by a whole converged warp, with one answer for all lanes.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort)
{
    return __all_sync(0xffffffffu, mbar_wait_hot(bar, parity, abort));
}

// As mbar_wait, but for copies and tensor-core work already in flight, which
// have to land before the CTA may leave: goes on when *abort is raised.
__device__ __forceinline__ bool mbar_wait_landed(uint64_t* bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(p) :: "memory");
    return p != 0;
}

// Fetches the descriptor itself (it lies in the kernel's parameters).
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Brings a tile into L2 only.  L2 is where all SMs and copies see memory, so
// this may run before griddep_wait() on data that an earlier kernel writes.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t c0, int32_t c1)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                 ::"l"(map), "r"(c0), "r"(c1) : "memory");
}

// ------------------------------------------------------------------ clusters

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of every CTA of the cluster arrives, and waits for the others.
// Relaxed: it orders no memory (a release would first wait for all accesses of
// the thread, about 1000 cycles); what crosses CTAs before it has to be waited
// for on mbarriers, or be ordered by the fence after their initialisation.
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

// The same with a release: also what the threads did to another CTA's shared
// memory (arrivals on its barriers) has happened there.  For the last meeting
// of a cluster, after which a CTA's shared memory may belong to another.
__device__ __forceinline__ void cluster_sync_release()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    cluster_wait();
}

// Address of the cluster's CTA `rank` that corresponds to this CTA's own
// shared-memory address.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Copies this CTA's shared memory into another's of the cluster and counts the
// bytes on a barrier there (16-byte aligned addresses and size; `dst` and `bar`
// are shared::cluster addresses of the same CTA).
__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "r"(src), "r"(bytes), "r"(bar) : "memory");
}

// ------------------------------------------------------------------ CTA pairs
// cta_group::2: two CTAs of a cluster work on one tensor-core product.  Each
// holds half of A's rows, half of B's rows and the accumulator lanes of its
// own half of A; one thread of the pair's first CTA issues the products.

// 2-D tile load into this CTA's shared memory that counts its bytes on a
// barrier of either CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                                 int32_t c1)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                 " [%0], [%1, {%3, %4}], [%2];"
                 ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(slot)), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tmem_relinquish_pair()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tc_mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// Arrive once on the barrier at this offset in both CTAs of the pair when the
// products issued so far by this thread have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

// Arrive on a barrier of another CTA of the cluster (a shared::cluster address).
// It releases within the CTA only: at cluster scope it would wait for the
// thread's outstanding accesses to memory, which took the epilogue of a
// projection's tile 3000 cycles.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

}  // namespace af
