// Host helpers of the entry points that launch one kernel family each
// (norm.cu, quant.cu, grouped.cu): pointer checks and a launch with
// programmatic stream serialisation (the kernel starts its prologue while the
// previous kernel of the stream drains, and waits for it before it reads).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "coli_moe.h"

namespace coli {

inline bool ptr_aligned(const void* p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;  // NULL counts as aligned
}

inline bool valid_dtype(int d) { return d == COLI_OUT_F32 || d == COLI_OUT_BF16; }

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
