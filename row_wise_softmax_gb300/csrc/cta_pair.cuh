// Primitives of a thread-block cluster of two CTAs that share tcgen05
// products (cta_group::2): the even CTA issues a product of 256 rows, of which
// each CTA holds 128 in its own shared and tensor memory, and each CTA holds
// half of the B operand.  The forms for a CTA on its own (CG = 1) sit beside.
#pragma once

#include "tcgen05.cuh"

#include <cudaTypedefs.h>

namespace rwsm {

template <int CG>
__device__ __forceinline__ uint32_t cta_rank()
{
    if constexpr (CG == 1)
        return 0;
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// All threads of the cluster (CG = 1: of the CTA).
template <int CG>
__device__ __forceinline__ void group_sync()
{
    if constexpr (CG == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The cluster-wide address of a shared-memory address in the even CTA.
template <int CG>
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr)
{
    if constexpr (CG == 1)
        return addr;
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

template <int CG>
__device__ __forceinline__ void mbar_arrive_leader(uint32_t addr)
{
    if constexpr (CG == 1)
        mbar_arrive(addr);
    else
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                     :: "r"(addr) : "memory");
}

// mbar_wait_bounded for a phase that threads of the other CTA complete too.
template <int CG>
__device__ __forceinline__ bool mbar_wait_group(uint32_t bar, uint32_t parity)
{
    if constexpr (CG == 1)
        return mbar_wait_bounded(bar, parity);
    unsigned long long t0 = 0;
    for (uint32_t it = 0; it < (1u << 30); ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok)
            return true;
        const unsigned long long now = global_ns();
        if (it == 0)
            t0 = now;
        else if (now - t0 > kWaitLimitNs)
            return false;
    }
    return false;
}

template <int CG>
__device__ __forceinline__ void tmem_alloc_group(uint32_t dst_smem, uint32_t ncols)
{
    if constexpr (CG == 1) {
        tmem_alloc(dst_smem, ncols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(dst_smem), "r"(ncols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_dealloc_group(uint32_t taddr, uint32_t ncols)
{
    if constexpr (CG == 1)
        tmem_dealloc(taddr, ncols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     :: "r"(taddr), "r"(ncols) : "memory");
}

template <int CG>
__device__ __forceinline__ void umma_f16_group(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 1)
        umma_f16(d_tmem, a_desc, b_desc, idesc, accumulate);
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                     : "memory");
}

template <int CG>
__device__ __forceinline__ void umma_f16_ta_group(uint32_t d_tmem, uint32_t a_tmem,
                                                  uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate)
{
    if constexpr (CG == 1)
        umma_f16_ta(d_tmem, a_tmem, b_desc, idesc, accumulate);
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// Commit to the barrier at this offset in both CTAs.
template <int CG>
__device__ __forceinline__ void umma_commit_group(uint32_t bar)
{
    if constexpr (CG == 1)
        umma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;"
                     :: "r"(bar), "h"(static_cast<unsigned short>(3)) : "memory");
}

// Tensor-map copy of a 3-D box into this CTA, completing on a barrier that
// may be the even CTA's.
template <int CG>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];"
            :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
            :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

}  // namespace rwsm
