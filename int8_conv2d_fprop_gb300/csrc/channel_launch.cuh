// channel_launch.cuh -- host-side launch helpers of the channel operators.
#pragma once

#include <cuda_runtime.h>

#include "channel.h"

namespace i8c {

// Every launch may start while the stream's previous kernel ends (it waits
// for that kernel before it touches memory; none of these kernels uses
// non-coherent loads, which would want their data final at the start).
template <typename... P, typename... A>
inline bool launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// Whether a row can be read in 16-byte vectors.
inline bool vector_rows(const MatRef &m) {
    if (!m.p) return true;
    return m.cs <= 1 && (uintptr_t)m.p % 16 == 0 && m.rs * channel_elem_size(m.dtype) % 16 == 0;
}

}  // namespace i8c
