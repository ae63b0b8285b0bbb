// Programmatic dependent launch of kernels that take their place while the stream's previous
// kernel drains: a launch of its own costs about 2 us between two kernels, as much as the
// smallest of them run.  A kernel launched this way calls depend_wait() in every CTA before
// its first access of global memory: it returns once the previous kernel has completed and
// its writes are visible, so nothing that an earlier kernel still uses is touched.  Its pointers
// are not __restrict__: that would promise that nobody else writes what the kernel reads while
// it lives, and let the compiler move those loads above the wait.  The
// kernel behind it may take its place the same way once every CTA of this one has called
// depend_next() or ended.  That call stands near a CTA's end: CTAs that come to wait among
// running ones fill the SMs unevenly (at the start of the decode kernel it cost 3 of 14 us).
// A kernel or copy that is launched plainly waits as always.
#pragma once

#include <cuda_runtime.h>

namespace hga {

__device__ __forceinline__ void depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void depend_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches in clusters of `cluster` CTAs along x (1: none).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster,
                             cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace hga
