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

// Loads of what a kernel before wrote, where this one starts before that ends: of memory as it
// is after the wait for it, so none by way of the caches for what nobody writes (those are
// defined where memory stays as it is for the kernel's life, which began before the wait), and
// volatile where they are not plain ones, so that none is moved before the wait.
// From L2.
template <typename T> __device__ __forceinline__ T load_l2(const T *p) {
    static_assert(sizeof(T) == 4 || sizeof(T) == 8, "a word or two");
    T r;
    if constexpr (sizeof(T) == 4) {
        uint32_t w;
        asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(w) : "l"(p));
        memcpy(&r, &w, 4);
    } else {
        uint2 w;
        asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p));
        memcpy(&r, &w, 8);
    }
    return r;
}
// What is not read again.
__device__ __forceinline__ uint4 load_once(const uint4 *p) {
    uint4 r;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Elements of 16 bytes.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

// Elements e .. e + E - 1 of a dense line at p + e (element e itself there), of which
// `room` are there, whatever p's alignment: from the two aligned 16-byte pieces that
// hold them, where both lie inside the line, else one by one.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T *line, int64_t e, int64_t length) {
    constexpr int E = kVec<T>;
    const T *p = line + e;
    const uint32_t off = (uint32_t)(uintptr_t)p & 15u;
    if (off == 0) return load_once((const uint4 *)p);
    const uint4 *lo = (const uint4 *)((uintptr_t)p - off);
    if ((const char *)lo >= (const char *)line && (const char *)(lo + 2) <= (const char *)(line + length)) {
        const uint4 u = lo[0], v = lo[1];
        uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        if (off & 8) w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = w[6], w[5] = w[7];
        if (off & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5];
        if constexpr (sizeof(T) == 2) {
            const uint32_t bits = (off & 2) * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    alignas(16) T t[E];
#pragma unroll
    for (int i = 0; i < E; ++i) t[i] = p[i];
    return *(const uint4 *)t;
}

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
