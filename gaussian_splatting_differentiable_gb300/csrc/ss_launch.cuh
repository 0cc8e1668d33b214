// Launches that begin while the kernel before them in the stream ends
// (programmatic dependent launch): the start of one and the end of the other
// overlap, and what the later kernel reads of the earlier one's it reads
// after wait_for_previous().
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace ss {

// Until the kernel before this one has ended and its writes are visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel after this one may be started (once every CTA has said so).
__device__ __forceinline__ void start_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// kernel<<<grid, threads, smem, s>>>(args...), allowed to start before the
// kernel before it in the stream has ended.  Every path of the kernel that
// touches memory calls wait_for_previous() first.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace ss
