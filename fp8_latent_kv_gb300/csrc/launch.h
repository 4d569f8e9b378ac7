// launch.h -- a kernel launched as a programmatic dependent of the one before it on its stream: it may start while that one
// ends, and calls sm100::grid_dependency_wait() before it touches memory.  What it reads may be written while it already runs, so none of
// its loads is a read-only one (no __ldg, no const __restrict__ parameter): those ask for memory that stays as it is all the
// kernel's life, and may be moved ahead of the wait.
#pragma once

#include <cuda_runtime.h>

namespace kv8 {

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace kv8
