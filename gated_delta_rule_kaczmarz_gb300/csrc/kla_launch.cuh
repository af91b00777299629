// Launches whose setting up runs under the end of the kernel before them in the
// stream (programmatic dependent launch).  Such a kernel begins with
// after_previous() in every thread, before it reads or writes memory: it waits for
// the kernel before to be complete, and as that one did the same, for all before it.
// A kernel that calls let_next_start() allows the next such launch from then on; its
// blocks start once all blocks of this one have.
#pragma once

#include <cuda_runtime.h>

namespace kla {

__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename Arg>
cudaError_t launch_next(void (*kernel)(const Arg), unsigned grid, unsigned block, size_t smem, int cluster,
                        const Arg &arg, cudaStream_t s) {
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, arg);
}

}  // namespace kla
