// sv_tc.cuh -- the tensor-core kernels' primitives (sm_100a): mbarriers with
// bounded waits, tiled TMA copies, shared-memory matrix descriptors, TMEM reads.
#pragma once

#include <cuda.h>  // CUtensorMap
#include <stdint.h>

#include "sv_common.cuh"

namespace sv {

__device__ __forceinline__ uint32_t lr_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void lr_mbar_init(uint64_t* bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(lr_smem(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void lr_expect_tx(uint64_t* bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(lr_smem(bar)), "r"(bytes) : "memory");
}

// One poll that may suspend the thread for up to kLrPollNs while the phase is
// still open (it returns as soon as the phase completes), so waiting warps take
// no issue slots from the producer and the MMA thread.
constexpr unsigned kLrPollNs = 20000;
constexpr unsigned kLrPolls = 200000;  // with the suspension: seconds, not hours

__device__ __forceinline__ bool lr_try_wait(uint64_t* bar, unsigned parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(lr_smem(bar)), "r"(parity), "r"(kLrPollNs)
        : "memory");
    return ok != 0;
}

// Whether the phase with this parity has completed, without suspending.
__device__ __forceinline__ bool lr_test(uint64_t* bar, unsigned parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(lr_smem(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for the phase with this parity; false (after raising the flags) if it did
// not complete within kLrPolls polls, or another role of the CTA already gave up.
__device__ __forceinline__ bool lr_wait(uint64_t* bar, unsigned parity, volatile int* abort, int* err)
{
    for (unsigned i = 0; i < kLrPolls; ++i) {
        if (lr_try_wait(bar, parity)) return true;
        if ((i & 63u) == 63u && *abort) return false;
    }
    *abort = 1;
    if (err) atomicExch(err, 1);
    return false;
}

// shared -> global tensor store of one staged chunk; rows and columns past the
// tensor's extent are not written
__device__ __forceinline__ void lr_tma_store_2d(const CUtensorMap* map, const void* src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"((uint64_t)map),
                 "r"(lr_smem(src)), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void lr_tma_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            lr_smem(dst)),
        "l"((uint64_t)map), "r"(lr_smem(bar)), "r"(x), "r"(y)
        : "memory");
}

// Shared-memory matrix descriptor of a K-major tile written by TMA with the
// 128-byte swizzle: rows of 128 bytes, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t lr_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu)   // start address, 16-byte units
           | ((uint64_t)1 << 16)                 // leading byte offset (unused for swizzled K-major)
           | ((uint64_t)(1024 >> 4) << 32)       // stride byte offset: 8 rows x 128 bytes
           | ((uint64_t)1 << 46)                 // descriptor version (sm_100)
           | ((uint64_t)2 << 61);                // layout: 128-byte swizzle
}

__device__ __forceinline__ void lr_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(lr_smem(bar))
                 : "memory");
}

__device__ __forceinline__ void lr_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void lr_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void lr_tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void lr_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(lr_smem(bar)) : "memory");
}

}  // namespace sv
