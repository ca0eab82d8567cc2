// Clusters and CTA pairs: barriers across the CTAs of a cluster, tcgen05 products of a pair of CTAs
// (cta_group::2), and the bounded wait of their pipelines (inline PTX; sm_100-family).
#pragma once

#include "tcgen05.cuh"

namespace oasr {

// All threads of the cluster; shared-memory accesses before it happen before those behind it.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// What CTA `rank` of the cluster has in shared memory where `addr` is here.
__device__ __forceinline__ float ld_shared_cluster(uint32_t addr, uint32_t rank)
{
    float v;
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_shared_cluster4(uint32_t addr, uint32_t rank)
{
    float4 v;
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

// Releases in the cluster what happened to this CTA's shared memory before it; a release of all memory at that
// scope waits for global memory's writes as well (0.6 us measured).
__device__ __forceinline__ void fence_release_smem_cluster()
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}

// Arrive on CTA `rank`'s barrier at the address that `bar` has here; orders no memory access by itself.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar, uint32_t rank)
{
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar),
                 "r"(rank)
                 : "memory");
}

// mbar_try_wait_sleep with acquire semantics in the cluster: for a barrier that another CTA's threads arrive on.
__device__ __forceinline__ bool mbar_try_wait_sleep_cluster(uint32_t bar, uint32_t parity, uint32_t hint_ns)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(hint_ns)
        : "memory");
    return done != 0;
}

// As wait_or_abort, with the timer, slow to read, left alone until a first sleep has run out (CLUSTER: acquires
// in the cluster).
template <bool CLUSTER = false>
__device__ __forceinline__ bool sleep_or_abort(uint32_t bar, uint32_t parity, volatile int* abort)
{
    // suspended until the phase completes, for 20 us at most between the checks below
    auto wait = [&] { return CLUSTER ? mbar_try_wait_sleep_cluster(bar, parity, 20000u) : mbar_try_wait_sleep(bar, parity, 20000u); };
    if (wait()) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (wait()) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
}

// A pair of CTAs (cta_group::2, issued by the even one): D has A's rows of each CTA in that CTA's TMEM, B's rows
// are half in one's shared memory and half in the other's, at the same offsets.
__device__ __forceinline__ void umma_ss_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, int acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a), "l"(b), "r"(id), "r"(acc));
}

// Arrives at `bar`'s offset in both CTAs of the pair.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Ask the hardware for the next CTA of the grid that has not started, to do its work here: the answer (16 bytes)
// goes to `to`, counted on `bar`.
__device__ __forceinline__ void ask_next(uint32_t to, uint32_t bar)
{
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to), "r"(bar)
                 : "memory");
}
// Its index; -1 when every CTA has started (no more is asked then).
__device__ __forceinline__ int next_cta(uint32_t from)
{
    uint32_t x, got;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tmov.u32 %0, 0;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %1, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, r;\n\t}"
        : "=&r"(x), "=&r"(got)
        : "r"(from)
        : "memory");
    return got ? static_cast<int>(x) : -1;
}

#define OASR_TMEM_LD16(taddr, r)                                                                   \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"  \
                 "%12,%13,%14,%15}, [%16];"                                                        \
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),          \
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),        \
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])                               \
                 : "r"(taddr))

#define OASR_TMEM_ST8(taddr, r)                                                                    \
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),         \
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])      \
                 : "memory")

}  // namespace oasr
