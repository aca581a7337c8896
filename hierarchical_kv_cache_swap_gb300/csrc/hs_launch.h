// Launches of the latent kernels as programmatic dependents (host code).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace hs {

// Launches `kernel`, allowed to begin before the kernel ahead of it on the stream is done: the
// kernel waits for that itself before it reads or writes anything.
template <class... Params, class... Args>
cudaError_t launch_dependent(cudaStream_t stream, dim3 grid, int threads, size_t smem, void (*kernel)(Params...), const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace hs
