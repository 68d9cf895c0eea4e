// chain.h -- launches of kernels that follow one another on a stream.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace txl {

// Kernels of one call are launched so that a kernel's blocks may be set up
// while the kernel before it on the stream drains: each kernel lets its
// successor do so at once, and waits for its predecessor's memory before it
// touches any.  A kernel is thus alive while others still write what it will
// read: no load of theirs goes the way of memory that stays as it is (__ldg,
// const __restrict__), which might be taken from before the wait.
__device__ __forceinline__ void chain_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... K, typename... A>
cudaError_t chain_launch(void (*kernel)(K...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                         cudaStream_t s, const A &...args)
{
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace txl
