// tw_kv.cuh — what the kernels of the paged key-value cache share.
#pragma once

#include <cstdint>
#include <mutex>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tw_device.cuh"
#include "tw_internal.h"

namespace tw {

// Run `ask` (what a kernel wants beyond the defaults: an attribute of a
// function) once per device and context: after a device reset, whose context
// has another id, it is asked again.  One cache per call site.
template <class F>
cudaError_t ask_once(F ask)
{
    static std::mutex mu;
    static unsigned long long asked[SymbolCache::kDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long id = context_id();
    std::lock_guard<std::mutex> lk(mu);
    if (dev < SymbolCache::kDevices && id && asked[dev] == id)
        return cudaSuccess;
    e = ask();
    if (e == cudaSuccess && dev < SymbolCache::kDevices)
        asked[dev] = context_id();
    return e;
}

}  // namespace tw
