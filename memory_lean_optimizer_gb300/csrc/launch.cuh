// launch.cuh -- programmatic dependent launch within a call.
#pragma once

#include <cuda_runtime.h>

namespace lmo {

// Programmatic dependent launch: a kernel starts while its predecessor on the stream drains and waits here
// before it touches memory; each lets its own successor start only after that wait, so what lies
// further back is complete too.  (A predecessor that does not let it start early, of whatever
// origin, is simply waited for.)
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_sync() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    pdl_release();
}

// Launches a kernel that waits for its predecessor itself (pdl_sync), as clusters of `cta`.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cta, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cta;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cta > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace lmo
