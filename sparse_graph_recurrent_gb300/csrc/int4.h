// Pieces that the two products with 4-bit weights share: their arguments, the way
// of weights and scales into a warp's hands, and weights as 16-bit floats.
#pragma once

#include <cuda.h>

#include <cstring>

#include "ck_types.h"

namespace ck {

struct MatvecArgs {
    const void *x;
    int64_t dtype, M, K, x_stride;
    const uint8_t *q;
    int64_t V, q_pitch;
    const void *scales;
    int scale_dtype;
    int64_t s_stride;
    const uint8_t *zeros;
    int64_t z_stride;
    const float *bias;
    void *y;
    int64_t y_stride;
    float *partial;  // slots of sums that cross CTAs or slabs
};

constexpr int kTileRows = 32;               // weight rows of a unit
constexpr int kChunk = 256;                 // columns of a unit
constexpr int kUnitBytes = kTileRows * kChunk / 2;
constexpr size_t kSmemMost = 232448 - 1024;  // of a CTA, less what is not dynamic

// a / b, in 32 bits where that does: a 64-bit division costs ten times as much
__host__ __device__ inline int64_t quotient(int64_t a, int64_t b) {
    return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// n things dealt to `to` owners in runs that differ by one at most
struct Deal {
    int64_t each, more;
    static __host__ __device__ Deal of(int64_t n, int64_t to) {
        const int64_t q = quotient(n, to);
        return Deal{q, n - q * to};
    }
    __host__ __device__ int64_t first(int64_t owner) const { return owner * each + (owner < more ? owner : more); }
    __host__ __device__ int64_t owner(int64_t i) const {
        const int64_t big = more * (each + 1);
        return i < big ? quotient(i, each + 1) : more + quotient(i - big, each);
    }
};

__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// q - z of a word's eight nibbles, as pairs (0, 4), (1, 5), (2, 6), (3, 7), times
// 2^-6 (bf16) or 2^-9 (fp16).  Alone in the low bits of a bf16 a nibble is the
// number q 2^-133, in the next place 16 q 2^-133 (fp16: 2^-24), exactly: so an AND
// and a multiply-add, whose factor evens out the places, give the exact difference,
// and of the four pairs two cost a shift.
template <bool HALF> struct Nibble {
    static constexpr uint32_t kLow = HALF ? 0x78007800u : 0x7f007f00u;   // 2^15, 2^127
    static constexpr uint32_t kHigh = HALF ? 0x68006800u : 0x7d007d00u;  // 2^11, 2^123
    static constexpr float kBack = HALF ? 512.f : 64.f;
    static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        if constexpr (HALF)
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        else
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    // -z, likewise, of byte i of four packed zero points
    static __device__ __forceinline__ uint32_t minus(uint32_t packed, int i) {
        return fma(__byte_perm(packed, 0u, 0x4040u | i | i << 8), kLow ^ 0x80008000u, 0u);
    }
    static __device__ __forceinline__ void pairs(uint32_t w, uint32_t z, uint32_t (&v)[4]) {
        const uint32_t w8 = w >> 8;
        v[0] = fma(w & 0x000f000fu, kLow, z);
        v[1] = fma(w & 0x00f000f0u, kHigh, z);
        v[2] = fma(w8 & 0x000f000fu, kLow, z);
        v[3] = fma(w8 & 0x00f000f0u, kHigh, z);
    }
};

// Three bf16 parts of a 32-bit float: each takes the top eight bits of what is
// left.  Cutting keeps the first part of a large number finite; what is not finite
// goes whole into the first part.
__device__ __forceinline__ void split3(float v, uint16_t (&part)[3]) {
    const uint32_t b = __float_as_uint(v);
    const bool odd = (b & 0x7f800000u) == 0x7f800000u;
    const uint32_t nan = (b & 0x007fffffu) && odd ? 0x00400000u : 0u;  // NaN stays NaN when cut
    const uint32_t h = (b | nan) & 0xffff0000u;
    const float r = odd ? 0.f : v - __uint_as_float(h);
    const uint32_t m = __float_as_uint(r) & 0xffff0000u;
    const float l = r - __uint_as_float(m);
    part[0] = (uint16_t)(h >> 16);
    part[1] = (uint16_t)(m >> 16);
    part[2] = (uint16_t)(__float_as_uint(l) >> 16);
}

// Eight numbers of a row of x from column k on, zeros past K.
template <typename T>
__device__ __forceinline__ void load8(const MatvecArgs &a, int64_t m, int64_t k, T (&v)[8]) {
    const T *src = (const T *)a.x + m * a.x_stride + k;
    if (k + 8 <= a.K && ((uintptr_t)src & 15) == 0) {
        constexpr int kVec = (int)sizeof(T) / 2;
        uint4 t[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) t[i] = ((const uint4 *)src)[i];
        memcpy(v, t, sizeof(t));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < a.K ? src[e] : from_float<T>(0.f);
    }
}

// Bounded wait on a shared-memory barrier's phase.  Time is the SM's clock: the
// global one takes longer to read than most waits last.
struct Waiter {
    volatile int *dead;
    long long limit;  // cycles
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t phase) const {
        long long began = 0;
        for (int i = 1;; ++i) {
            uint32_t done;
            asm volatile(
                "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                : "=r"(done) : "r"(bar), "r"(phase) : "memory");
            if (done) return true;
            if ((i & 63) == 0) {
                if (*dead) return false;
                const long long now = clock64();
                if (began == 0) began = now;
                if (now - began > limit) {
                    *dead = 1;
                    return false;
                }
            }
        }
    }
};

__device__ __forceinline__ void barrier_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// One thread of the warp, which runs as one, has a box of the weights copied to shared
// memory at dst; `bar` is told of its bytes.
__device__ __forceinline__ void copy_box(const CUtensorMap &map, int byte, int row, uint32_t dst, uint32_t bar,
                                         uint32_t bytes) {
    asm volatile(
        "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%4], %5;\n"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
        "l"(&map), "r"(byte), "r"(row), "r"(bar), "r"(bytes)
        : "memory");
}

__device__ __forceinline__ float scale_value(uint32_t raw, int dtype) {
    if (dtype == CK_F32) return __uint_as_float(raw);
    if (dtype == CK_BF16) return __uint_as_float(raw << 16);
    return __half2float(__ushort_as_half((unsigned short)raw));
}

// Scales and zero points, read eight groups of a tile's 32 rows at a time: lane l
// of load i takes group l % 8 of row 4 i + l / 8, so that a load touches four rows'
// sectors and not 32.  Kept as they come from memory until the groups are begun (a
// conversion would wait for the loads), then left in shared memory as [row][PITCH] scales and
// [row][8] zero points.
template <int PITCH> struct ScaleReader {
    uint32_t s[8], z[8];
    int tile, eight;  // what s and z hold
    __device__ __forceinline__ void load(const MatvecArgs &a, int tile_, int eight_, int groups) {
        tile = tile_;
        eight = eight_;
        const int lane = threadIdx.x & 31, g = 8 * eight + (lane & 7), v = tile * kTileRows + (lane >> 3);
        const int rows = g < groups ? (int)a.V - v : 0;  // row 4 i is there if 4 i < rows
        if (a.scale_dtype == CK_F32) {
            const uint32_t *p = (const uint32_t *)a.scales + v * a.s_stride + g;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = 4 * i < rows ? p[4 * i * a.s_stride] : 0u;
        } else {
            const uint16_t *p = (const uint16_t *)a.scales + v * a.s_stride + g;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = 4 * i < rows ? p[4 * i * a.s_stride] : 0u;
        }
        if (a.zeros) {
            const uint8_t *p = a.zeros + v * a.z_stride + g;
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = 4 * i < rows ? p[4 * i * a.z_stride] : 8u;
        }
    }
    // A line of each row towards L2, a row to a lane, once for each 128 bytes: a load a
    // unit ahead alone waits for memory.
    static __device__ __forceinline__ void ahead(const MatvecArgs &a, int tile, int eight, int groups, bool start) {
        const int v = tile * kTileRows + (threadIdx.x & 31), g = 8 * eight;
        if (v >= (int)a.V || g >= groups) return;
        const int size = a.scale_dtype == CK_F32 ? 4 : 2;
        const char *p = (const char *)a.scales + (v * a.s_stride + g) * size;
        if (start || ((uintptr_t)p & 127) < 8 * size) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
        if (a.zeros) {
            const uint8_t *q = a.zeros + v * a.z_stride + g;
            if (start || ((uintptr_t)q & 127) < 8) asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
        }
    }
    __device__ __forceinline__ void leave(const MatvecArgs &a, float *scales, uint8_t *zeros) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            scales[(4 * i + (lane >> 3)) * PITCH + (lane & 7)] = scale_value(s[i], a.scale_dtype);
            zeros[32 * i + lane] = a.zeros ? (uint8_t)(z[i] & 15) : (uint8_t)8;
        }
    }
};


__device__ __forceinline__ void store_y(const MatvecArgs &a, int64_t m, int64_t v, float sum) {
    sum += a.bias ? a.bias[v] : 0.f;
    const int64_t at = m * a.y_stride + v;
    if (a.dtype == CK_F32)
        ((float *)a.y)[at] = sum;
    else if (a.dtype == CK_BF16)
        ((__nv_bfloat16 *)a.y)[at] = __float2bfloat16_rn(sum);
    else
        ((__half *)a.y)[at] = __float2half_rn(sum);
}

// Weights as a two-dimensional array of bytes, copied `rows` rows by 128 bytes at a
// time with 16-byte pieces exchanged by the row (the 128-byte swizzle); zeros past its ends.
inline cudaError_t weight_map(const MatvecArgs &a, int rows, CUtensorMap *map) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> known{nullptr};
    Encode encode = known.load();
    if (!encode) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
        known = encode = (Encode)f;
    }
    const cuuint64_t size[2] = {(cuuint64_t)((a.K + 1) / 2), (cuuint64_t)a.V}, pitch[1] = {(cuuint64_t)a.q_pitch};
    const cuuint32_t box[2] = {kChunk / 2, (cuuint32_t)rows}, one[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)a.q, size, pitch, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// The product for more columns than k_matvec takes (int4_wide.cu): rows of x in one
// call, the workspace that a call needs, and the call.
int64_t wide_rows(int64_t dtype);
size_t wide_workspace(int64_t dtype, int64_t rows, int64_t K, int64_t V, int sms);
cudaError_t launch_wide(const MatvecArgs &a, int64_t group, void *workspace, int sms, cudaStream_t stream);

}  // namespace ck
