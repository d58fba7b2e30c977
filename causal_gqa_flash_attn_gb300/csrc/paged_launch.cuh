// paged_launch.cuh -- launches that overlap the end of the kernel before them in
// the stream (programmatic dependent launch). The kernel's blocks may be placed
// while that one drains; its first statement is wait_for_stream(), behind which
// everything before it is done and visible.
#pragma once

#include <cuda_runtime.h>

namespace fa {

__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// What the kernel before may have written is read by ordinary loads: read-only ones
// (ld.global.nc) want memory that nothing writes while the kernel is there, and it is
// there, waiting, while the other one writes.
template <typename T>
__device__ __forceinline__ T load(const T *p) {
    return *p;
}

// A launch in the middle of a stream costs about 2 us less than a plain one (32 tokens'
// rotation 4.2 -> 2.3 us, 12 requests' append and gather 104.5 -> 99.5).
template <typename Args>
inline cudaError_t launch_after(void (*kernel)(Args), dim3 blocks, int threads, size_t smem,
                                cudaStream_t stream, const Args &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = blocks;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace fa
