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

__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
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
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

__device__ __forceinline__ void tma_2d(void* dst, const void* map, int c0, int c1, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const void* map, int c0, int c1, int c2,
                                       uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

}  // namespace tc
}  // namespace coli
