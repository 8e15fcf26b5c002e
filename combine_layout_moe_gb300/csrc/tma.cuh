// Bulk asynchronous copies (the TMA engine's non-tensor form) and mbarriers,
// as inline PTX for sm_90 and later.  Every wait is bounded: a wait that gives
// up reports MOE_ERRBIT_TIMEOUT through the caller instead of spinning forever.
#pragma once

#include <cstdint>

namespace moe {

// A wait gives up after this much wall-clock time (the device's global
// nanosecond timer), whatever the hardware does inside each try_wait.
constexpr uint64_t MBAR_TIMEOUT_NS = 1000000000ull;

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Makes barrier initialisation visible to the async (bulk-copy) proxy.
__device__ __forceinline__ void mbar_fence_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Waits until the phase with the given parity has completed; false once
// MBAR_TIMEOUT_NS has passed.  The caller must never be two or more phases
// ahead of the barrier (parity alone cannot tell those apart): every pipeline
// here gives each stage a single consumer that waits on its phases in order.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (global_ns() - t0 > MBAR_TIMEOUT_NS)
            return false;
    }
}

// Whether the phase has completed, at once: for a look ahead whose answer is not needed
// yet.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// mbar_try_wait that may leave the thread suspended for longer (up to `ns`), until
// the phase completes: a warp that waits then takes no issue slots from the others.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(ns)
        : "memory");
    return done != 0;
}

// mbar_wait in such tries, for waits that follow each other closely.
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity)
{
    constexpr uint32_t TRY_NS = 1000000;
    if (mbar_try_wait_for(bar, parity, TRY_NS))
        return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait_for(bar, parity, TRY_NS))
        if (global_ns() - t0 > MBAR_TIMEOUT_NS)
            return false;
    return true;
}

// This thread's warp in its CTA, in a form that the compiler knows to be the same for
// the whole warp.
__device__ __forceinline__ int warp_index()
{
    return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
}

// The same for a whole warp, whose lanes agree on the answer; no wait at all once `ok`
// is false, which ends true as long as none has given up.  Loops around such waits run
// on in any case, doing nothing, so that their control does not depend on `ok` and
// their addresses and descriptors stay in uniform registers.
__device__ __forceinline__ void warp_wait(bool &ok, uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
        "TRY_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "vote.sync.all.pred p, p, 0xffffffff;\n\t"
        "@p bra.uni DONE_%=;\n\t"
        "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, %3;\n\t"
        "@q bra.uni TRY_%=;\n"
        "DONE_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(ok ? 256u : 0u)
        : "memory");
    if (done == 0 && ok)
        ok = __all_sync(0xffffffffu, mbar_wait_short(bar, parity));
}

// For two barriers; the answers of both first tries are awaited together.
__device__ __forceinline__ void warp_wait2(bool &ok, uint32_t bar_a, uint32_t parity_a,
                                           uint32_t bar_b, uint32_t parity_b)
{
    const bool a = mbar_try_wait(bar_a, parity_a), b = mbar_try_wait(bar_b, parity_b);
    if (__all_sync(0xffffffffu, a && b))
        return;
    warp_wait(ok, bar_a, parity_a);
    warp_wait(ok, bar_b, parity_b);
}

// One arrival for a whole warp, without a branch.
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(threadIdx.x & 31)
        : "memory");
}

// Global -> shared bulk copy of `bytes` (multiple of 16, both addresses
// 16-byte aligned); completion is counted on mbarrier `bar` as transaction bytes.
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void *src, uint32_t bytes,
                                         uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Shared -> global bulk copy, tracked by the issuing thread's bulk async-group.
__device__ __forceinline__ void bulk_s2g(void *dst, uint32_t src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
                 "r"(bytes)
                 : "memory");
}

// Orders this thread's earlier shared-memory accesses (and what it observed
// through mbarriers) before its later bulk-copy accesses to shared memory.
__device__ __forceinline__ void fence_proxy_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// Waits until at most N of this thread's committed bulk groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Waits until all of this thread's committed bulk groups have completed.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace moe
