// fp8z_launch.cuh -- launches whose blocks may be set up while the kernel before
// them in the stream still runs.
//
// A kernel launched this way starts with dependent_wait(): until it returns,
// the kernel before it may still be writing, and nothing is read or written.
// Its pointers carry no __restrict__: a load from memory promised to be constant
// might be moved before the wait.
// Each kernel then lets its own successor be set up.  A chain of short kernels
// loses the 1 to 2 us between two of them that way.
#pragma once

#include <utility>

#include <cuda_runtime.h>

#include "fp8z.h"

namespace fp8z {

__device__ __forceinline__ void dependent_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// cluster: blocks along x of a cluster, 0 where the kernel itself says how many.
template <typename... P, typename... A>
int launch_dependent_clusters(void (*kernel)(P...), int cluster, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              A&&... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(unsigned(threads));
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = cluster > 0 ? 2 : 1;
    if (cudaLaunchKernelEx(&c, kernel, static_cast<P>(std::forward<A>(args))...) == cudaSuccess) return FP8Z_OK;
    cudaGetLastError();                    // reported here, not by the next call that asks
    return FP8Z_ECUDA;
}

template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
    return launch_dependent_clusters(kernel, 0, grid, threads, smem, stream, std::forward<A>(args)...);
}

}  // namespace fp8z
