// Inline-PTX wrappers for the fifth-generation tensor cores with both operands
// in shared memory (128-byte swizzle), and for tensor-map loads.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "ptx.cuh"

namespace coli {
namespace tc {

// Shared-memory operand descriptors, 128-byte swizzle (rows of 128 bytes,
// atoms of 8 rows = 1024 bytes).
//   K-major: a row holds 128 bytes along the reduction; SBO is the step from 8
//   rows to the next 8, LBO is not used.
//   MN-major: a row holds 128 bytes along M (or N) at one reduction index;
//   SBO is the step from 8 reduction indices to the next 8, LBO the step from
//   64 elements of M (N) to the next 64.
__device__ __forceinline__ uint64_t desc_base(uint32_t lbo, uint32_t sbo) {
    return ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
           ((uint64_t)1 << 46)    // descriptor version for sm_100
           | ((uint64_t)2 << 61);  // 128-byte swizzle
}
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t saddr) {
    return base | (uint64_t)((saddr & 0x3FFFFu) >> 4);
}

// Instruction descriptor: fp32 accumulators, M rows, N columns; a/b_fmt: the
// operand formats of the kind; a/b_mn: 1 for an MN-major operand.
__device__ __forceinline__ uint32_t idesc(int M, int N, uint32_t fmt, uint32_t a_mn, uint32_t b_mn) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (a_mn << 15) | (b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <bool kFp8, int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
#define COLI_MMA(GROUP, KIND)                                                                \
    asm volatile(                                                                            \
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"                                    \
        "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d), \
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                          \
        : "memory")
    if constexpr (kFp8) {
        if constexpr (CTAS == 1) COLI_MMA("1", "f8f6f4");
        else COLI_MMA("2", "f8f6f4");
    } else {
        if constexpr (CTAS == 1) COLI_MMA("1", "f16");
        else COLI_MMA("2", "f16");
    }
#undef COLI_MMA
}

// Arrive on `bar` when the MMAs issued so far are done; with CTAS = 2 on the
// barrier at the same place in both CTAs of the pair.
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CTAS == 1)
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                bar)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
            ".b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
}

// The same on this CTA's barrier alone.
template <int CTAS>
__device__ __forceinline__ void commit_here(uint32_t bar) {
    if constexpr (CTAS == 1) commit<1>(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
}

template <int CTAS>
__device__ __forceinline__ void alloc(uint32_t* slot, uint32_t cols) {
    if constexpr (CTAS == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CTAS>
__device__ __forceinline__ void dealloc(uint32_t addr, uint32_t cols) {
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                     : "memory");
}

__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 16 consecutive columns of this warp's 32 lanes; ld_wait before use.
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
// The loaded registers pass through the wait, so that no use of them can be
// moved before it.
__device__ __forceinline__ void ld_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
}

// ---- tensor-map loads; `bar` is a shared::cluster address.  With CTAS = 2 the
// barrier may be the pair's other CTA's. ----
template <int CTAS>
__device__ __forceinline__ void tma_2d(uint32_t dst, const void* map, int c0, int c1, uint32_t bar) {
    if constexpr (CTAS == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tma_3d(uint32_t dst, const void* map, int c0, int c1, int c2,
                                       uint32_t bar) {
    if constexpr (CTAS == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
}

template <int CTAS>
__device__ __forceinline__ void tma_4d(uint32_t dst, const void* map, int c0, int c1, int c2, int c3,
                                       uint32_t bar) {
    if constexpr (CTAS == 1)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void prefetch_map(const void* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor-map stores (parts outside the tensor are not written).  What they
// write leaves L2 first: large results would push the operands out. ----
__device__ __forceinline__ void tma_store_3d(const void* map, const void* src, int c0, int c1,
                                             int c2, bool add) {
    if (add)
        asm volatile(
            "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group "
            "[%0, {%1, %2, %3}], [%4];" ::"l"(map),
            "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(src))
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint "
            "[%0, {%1, %2, %3}], [%4], %5;" ::"l"(map),
            "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(src)), "l"(policy_evict_first())
            : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The sources of all but the last N stores may be written again.
template <int N>
__device__ __forceinline__ void store_read_wait() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---- clusters of two CTAs ----
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// shared::cluster address of `p` in the CTA of rank `rank`
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// Arrive on a barrier of the cluster; the second form also releases this
// thread's writes to the other CTA (it waits for them, the first does not).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_release_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
// Bounded waits for a phase, false after `limit` ns.  A try suspends the
// thread until the phase completes or kTryNs have passed: threads that poll take
// issue slots from the two that feed the tensor cores (8192 x 6144 x 6144 bf16
// took 434 us with plain tries, 404 us so).
constexpr uint32_t kTryNs = 1000000;

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kTryNs)
        : "memory");
    return ok != 0;
}
// The same, and acquires what another CTA of the cluster released.
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kTryNs)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint64_t limit) {
    if (try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!try_wait(bar, parity))
        if (global_timer_ns() - t0 > limit) return false;
    return true;
}
// A whole warp's wait: its lanes go on or leave together.  A phase that this warp
// must still release stays complete, so lanes can differ only over the limit, and
// those that get there vote.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit) {
    const uint32_t at = smem_addr(bar);
    if (try_wait(at, parity)) return true;
    const unsigned lanes = __activemask();
    const uint64_t t0 = global_timer_ns();
    while (!__any_sync(lanes, try_wait(at, parity)))
        if (__any_sync(lanes, global_timer_ns() - t0 > limit)) return false;
    return true;
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit) {
    if (try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!try_wait_cluster(bar, parity))
        if (global_timer_ns() - t0 > limit) return false;
    return true;
}

// d[0..1] += v[0..1] * s as one packed instruction (half the issue slots, which
// the warps that feed the tensor cores share).
__device__ __forceinline__ void fma2(float* d, const uint32_t* v, float s) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\t"
        "fma.rn.f32x2 a, b, c, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(d[0]), "+f"(d[1])
        : "f"(__uint_as_float(v[0])), "f"(__uint_as_float(v[1])), "f"(s));
}

// Wait until at most N of this thread's latest cp.async groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Arrive on `bar` when this thread's cp.async copies so far are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// ---- register split between warpgroups ----
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace tc
}  // namespace coli
