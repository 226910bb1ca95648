// Launches of one call that follow each other on a stream: a kernel is launched while the one before it ends (programmatic
// dependent launch) and waits for its end itself, so its blocks' start is hidden behind it. Only ever behind a kernel
// of the same call, so that the inputs, which no kernel of the call writes, may be read before the wait. What the launch
// before wrote is read behind the wait and never through the read-only path (__ldg): that holds for memory that nobody
// writes while the reading kernel lives, and a chained kernel lives from before the wait on.
//
// A kernel that needs nothing of the one before it, and writes nothing that one reads, runs beside it: its last block waits
// at its end, so that when it has ended the other has (all blocks would hold their SMs until then). Whatever ended before
// the other passed its own wait at its start, or before a chain of such kernels began, has ended for it too, as nobody
// lets the next launch start before that; it reads what those wrote past L1 (__ldcg, tensor copies). Documented is what the
// launch that waits sees; for the one beside it this rests on an ended launch's writes being in L2, where it reads them.
#pragma once

#include <utility>

#include <cuda_runtime.h>

namespace sdm {

// all that the launch before wrote is there, and all that it reads may be written
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// the next launch may start its blocks as SMs become free
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

enum class Chain { behind, beside };
// at a kernel's start and end
__device__ __forceinline__ void chain_begin(Chain c) {
    if (c != Chain::beside) chain_wait();
    chain_next();
}
__device__ __forceinline__ void chain_end(Chain c) {
    if (c == Chain::beside && blockIdx.x == gridDim.x - 1) chain_wait();
}

template <typename... P, typename... A>
cudaError_t chain_launch(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchAttribute attribute{};
    attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attribute.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = st;
    config.attrs = &attribute;
    config.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&config, kern, std::forward<A>(args)...);
    if (e != cudaSuccess) cudaGetLastError();            // returned here, not found again by the next call
    return e;
}

}  // namespace sdm
