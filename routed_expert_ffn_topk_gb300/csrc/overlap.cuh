// Programmatic dependent launch of the 4-bit calls' kernels: a kernel's start (block
// launch, barriers, tensor memory) overlaps the end of the one before it in the
// stream. Between two small products, launched plainly, the device idles for
// about 4 us, which is as long as one of them runs.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace es {

// Every thread calls this before it touches memory that another kernel may write or
// read. The kernel after this one may then start, and this one continues once all
// those before it have ended and their writes are visible. What they may have
// written is read by ordinary loads, not by the read-only path (__ldg, or a const
// __restrict__ parameter): that path is defined only for memory which nothing
// writes while the kernel runs, and this one runs while they write.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}

inline cudaLaunchAttribute overlapped() {
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchAttribute at = overlapped();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace es
