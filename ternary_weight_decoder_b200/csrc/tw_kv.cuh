// tw_kv.cuh — the paged key-value cache as the kernels see it, and the
// conversions between its element types and fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "tw_device.cuh"
#include "tw_internal.h"

namespace tw {

// Element types of the pools.
template <int DT> struct KvElem;
template <> struct KvElem<TW_KV_BF16> { using type = __nv_bfloat16; };
template <> struct KvElem<TW_KV_F16> { using type = __half; };
template <> struct KvElem<TW_KV_I8> { using type = int8_t; };

__device__ __forceinline__ float kv_to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float kv_to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float kv_to_f32(int8_t v) { return (float)v; }

}  // namespace tw
