// Launch of a kernel as a programmatic dependent of the one before it on the
// stream.
#pragma once

#include <cuda_runtime.h>

namespace pkv_pdl {

// The kernel's CTAs may be resident before the kernel before it has ended; it
// has to wait_for_previous() before it touches memory.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), long long grid, int threads, int smem,
                             cudaStream_t stream, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Until the kernel before has completed and its writes are visible.
__device__ __forceinline__ void wait_for_previous()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Lets the kernel after this one become resident.
__device__ __forceinline__ void let_next_start()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace pkv_pdl
