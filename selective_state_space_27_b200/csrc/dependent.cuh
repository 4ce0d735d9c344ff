// Kernels that start before the one in front of them in the stream has ended
// (programmatic dependent launch).
#pragma once

#include <cuda_runtime.h>

namespace ms {

// Launch behind the previous kernel of the stream, without waiting for its end:
// the blocks start when all blocks of that kernel have called dependents_may_start
// or ended. What it writes may be used behind wait_for_previous.
template <typename... P>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             const P &...args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(static_cast<unsigned>(threads));
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = &early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

// The kernel behind this one may start: a block of it then waits on the device, so
// this is called where the space of this kernel's blocks is about to be free.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Until the kernel in front has ended and its writes are visible. No effect in a
// kernel launched the ordinary way.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace ms
