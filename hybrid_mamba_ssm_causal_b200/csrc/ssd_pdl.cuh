// ssd_pdl.cuh -- programmatic dependent launch of a call's kernels.
#pragma once

#include <cuda_runtime.h>

namespace ssd {

// A call's kernels follow one another by programmatic dependent launch: each lets its successor start
// (blocks placed, shared and tensor memory set up) as it starts itself, and waits for its predecessor
// before it touches global memory (the scan on CUDA cores lets it start later). Every block waits, so that
// a kernel's end implies its predecessor's. A call's first kernel is launched plainly.
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_follow()
{
    pdl_release();
    pdl_wait();
}
template <typename... P, typename... A>
cudaError_t pdl_launch(bool follows, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace ssd
