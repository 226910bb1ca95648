// Launches of one call that follow each other on a stream: a kernel is launched while the one before it ends (programmatic
// dependent launch) and waits for its end itself, so its blocks' start is hidden behind it. Only ever behind a kernel
// of the same call, so that the inputs, which no kernel of the call writes, may be read before the wait.
#pragma once

#include <utility>

#include <cuda_runtime.h>

namespace sdm {

// all that the launch before wrote is there, and all that it reads may be written
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// the next launch may start its blocks as SMs become free
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t chain_launch(bool chained, void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchAttribute attribute{};
    attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attribute.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = st;
    config.attrs = &attribute;
    config.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&config, kern, std::forward<A>(args)...);
}

}  // namespace sdm
