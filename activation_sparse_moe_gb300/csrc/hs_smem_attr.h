// Dynamic shared memory limits of the kernels (host code only: a test compiles
// it against a stand-in of the runtime).
#pragma once

#include <cuda_runtime.h>
#include <mutex>

#include "hs.h"

namespace hs_host {

// Raises a kernel's dynamic shared memory limit once per (kernel, device) and
// larger size: the attribute call is kept out of the per-call path (and out of
// stream capture after the first eager call).  A kernel has one entry, whatever
// sizes it is launched with.
inline int set_smem_attr(const void* fn, int bytes) {
    struct Entry { const void* fn; int dev; int bytes; };
    static Entry done[64];
    static int n_done = 0;
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return HS_ERR_CUDA;
    int i = 0;
    while (i < n_done && !(done[i].fn == fn && done[i].dev == dev)) ++i;
    if (i < n_done && done[i].bytes >= bytes) return HS_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return HS_ERR_CUDA;
    if (i < 64) done[i] = Entry{fn, dev, bytes};
    if (i == n_done && n_done < 64) ++n_done;
    return HS_OK;
}

}  // namespace hs_host
