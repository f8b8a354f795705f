// Element types of the readout operators (ck_dtype): conversions to and from
// the 32-bit floats that all of them compute in.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ck_internal.h"

namespace ck {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// Rounded once, to nearest even.
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

inline bool known_dtype(int64_t d) { return d == CK_F32 || d == CK_BF16 || d == CK_F16; }
inline size_t dtype_size(int64_t d) { return d == CK_F32 ? 4 : 2; }
// Whether p lies at a multiple of `bytes`, as a kernel's loads of that size need.
inline bool aligned(const void *p, size_t bytes) { return (uintptr_t)p % bytes == 0; }

// f((T *)nullptr) with T the element type of a (checked) ck_dtype.
template <typename F> auto with_dtype(int64_t d, F &&f) {
    switch (d) {
        case CK_BF16: return f((__nv_bfloat16 *)nullptr);
        case CK_F16: return f((__half *)nullptr);
        default: return f((float *)nullptr);
    }
}

// SMs of the current device, asked once for each (1 when it cannot be asked: the
// launch then reports why).
inline int device_sms() {
    constexpr int kMost = 64;
    static std::atomic<int> known[kMost];
    int dev = 0, sms = 1;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < kMost && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    if (dev < kMost) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// Allows a kernel `bytes` of dynamic shared memory, once for each device (`done`: a bit
// for each that has been told) and not on every launch.
inline cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace ck
