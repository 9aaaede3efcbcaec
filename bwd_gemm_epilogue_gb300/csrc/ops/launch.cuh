// launch.cuh -- what the operators' launches share on the host.
#pragma once

#include "../host.h"

namespace swiglu {

// Lets `kernel` be launched with `bytes` of dynamic shared memory, where the limit is lower: then it becomes the
// most that an SM has for it.  The limit is the kernel's, not the call's, so none that is lower may follow: another
// thread's call may be on its way to its launch.
inline cudaError_t allow_smem(const void* kernel, size_t bytes) {
    if (bytes <= 32 * 1024) return cudaSuccess;            // with the kernels' own arrays below the 48 KB that need no leave
    cudaFuncAttributes has;
    const cudaError_t e = cudaFuncGetAttributes(&has, kernel);
    if (e != cudaSuccess || (size_t)has.maxDynamicSharedSizeBytes >= bytes) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - (int)has.sharedSizeBytes);
}

}  // namespace swiglu
