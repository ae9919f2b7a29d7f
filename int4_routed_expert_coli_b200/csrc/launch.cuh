// Host helpers of the entry points that launch one kernel family each
// (norm.cu, quant.cu, grouped.cu): pointer checks and a launch with
// programmatic stream serialisation (the kernel starts its prologue while the
// previous kernel of the stream drains, and waits for it before it reads).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "coli_moe.h"

namespace coli {

inline bool ptr_aligned(const void* p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;  // NULL counts as aligned
}

inline bool valid_dtype(int d) { return d == COLI_OUT_F32 || d == COLI_OUT_BF16; }

// Lets `kernel` use up to `smem` bytes of dynamic shared memory: always the same
// number for a kernel, so that host threads cannot lower it under each other, and
// set once per device (`done`: one bit each).
inline cudaError_t allow_smem(const void* kernel, int smem, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

template <typename... P, typename... A>
cudaError_t launch_serialized(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace coli
