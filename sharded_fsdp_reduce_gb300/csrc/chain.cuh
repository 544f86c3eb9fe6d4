// chain.cuh -- chained launches: the kernels of one call that follow one
// another on a stream start while the one before them drains (programmatic
// stream serialization) and wait for its results themselves. Every kernel of
// a chain lets the next one start only after its own wait, so that a kernel
// that has started knows all work before its predecessor to be done. It waits
// before it touches memory, but for two that work beside their predecessor and
// wait last: the embedding gradient's zeros (fill_rows, behind the sort) and a
// teacher's entries beside a few rows' dot products (prepare_kernel, late). They
// may, since that predecessor is of the same call, has waited itself, and
// neither reads nor writes what they write, nor writes what they read. A kernel
// launched behind anything else has to wait first.
// Six kernels of 4 to 60 us each: 239 us a call without, 225 with.
#pragma once

#include "host.cuh"

namespace fsdp {

__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launch a kernel that waits for its predecessor on the stream itself
// (wait_previous) and may start before that one has ended.
template <class... Params, class... Args>
fsdp_status launch_chained(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                           Args &&...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = s;
    config.attrs = &attr;
    config.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&config, kernel, static_cast<Args &&>(args)...));
}

}  // namespace fsdp
