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

// Arrive on the even CTA's barrier.  What it announces lies in tensor memory
// and is ordered by tcgen05.wait and tcgen05.fence before it; no other memory
// is handed over, so the arrival and the waits keep the CTA scope (with
// .release.cluster and .acquire.cluster each wait that was already over cost
// about 250 cycles, each arrival several hundred).
template <int CG>
__device__ __forceinline__ void mbar_arrive_leader(uint32_t addr)
{
    if constexpr (CG == 1)
        mbar_arrive(addr);
    else
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(addr) : "memory");
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

// Products and commits, called by a whole warp in uniform control flow: the
// instruction itself is executed by the lane that elect.sync picks (the same
// one each time).  Their operands are warp-uniform registers, which uniform
// code holds already; issued from inside a one-lane branch they were moved
// there one by one, about 100 cycles a product beside busy warps.
template <int CG>
__device__ __forceinline__ void umma_f16_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// The same with A in tensor memory.
template <int CG>
__device__ __forceinline__ void umma_f16_ta_warp(uint32_t d_tmem, uint32_t a_tmem,
                                                 uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                     :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// Commit to the barrier at this offset in both CTAs.
template <int CG>
__device__ __forceinline__ void umma_commit_warp(uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
                     "[%0];\n\t}" :: "r"(bar) : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;\n\t}"
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

// Cluster launch control (sm_100): ask for a cluster of this grid that has not
// been launched yet, in its place.  The 16-byte answer arrives in both CTAs
// at this offset, with 16 bytes on the barrier at the other.
template <int CG>
__device__ __forceinline__ void clc_try_cancel(uint32_t answer, uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta"
                     ".mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                     :: "r"(answer), "r"(bar) : "memory");
    else
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta"
                     ".mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], [%1];"
                     :: "r"(answer), "r"(bar) : "memory");
}

// blockIdx.x of the first CTA of the cluster that an answer gave, -1 when it
// gave none (no cluster is left; nothing may be asked for after that).
__device__ __forceinline__ int64_t clc_first_cta(uint32_t answer)
{
    uint32_t given, x;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
                 "ld.shared.b128 r, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
                 : "=r"(given), "=r"(x) : "r"(answer) : "memory");
    return given ? static_cast<int64_t>(x) : -1;
}

}  // namespace rwsm
