// ck_int4_matvec and ck_int4_quantize: products of a few state rows with 4-bit
// weights, and the rounding that makes such weights.
#include "ck_types.h"

namespace ck {
namespace {

__device__ __forceinline__ float load_scale(const void *p, int dtype, int64_t i) {
    if (dtype == CK_F32) return ((const float *)p)[i];
    if (dtype == CK_BF16) return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
    return __half2float(((const __half *)p)[i]);
}

struct MatvecArgs {
    const void *x;
    int64_t M, K, x_stride;
    const uint8_t *q;
    int64_t V, q_pitch;
    const void *scales;
    int scale_dtype;
    int64_t s_stride;
    const uint8_t *zeros;
    int64_t z_stride;
    const float *bias;
    int group;
    void *y;
    int64_t y_stride;
};

// One warp per weight row and eight rows of x; a lane takes every 32nd word of
// eight weights.  A word lies in one group, as groups are multiples of eight.
constexpr int kRows = 8;
template <typename T> __global__ void __launch_bounds__(256) k_matvec(MatvecArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t v = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (v >= a.V) return;
    const T *x = (const T *)a.x;
    T *y = (T *)a.y;
    for (int64_t m0 = (int64_t)blockIdx.y * kRows; m0 < a.M; m0 += (int64_t)gridDim.y * kRows) {
        float acc[kRows] = {};
        for (int64_t k = 8 * lane; k < a.K; k += 8 * 32) {
            const int64_t g = k / a.group;
            const float s = load_scale(a.scales, a.scale_dtype, v * a.s_stride + g);
            const float z = a.zeros ? (float)(a.zeros[v * a.z_stride + g] & 15) : 8.f;
            const int n = a.K - k < 8 ? (int)(a.K - k) : 8;
            float w[8];
            for (int j = 0; j < n; ++j) {
                const uint8_t b = a.q[v * a.q_pitch + (k + j) / 2];
                w[j] = s * ((float)(j & 1 ? b >> 4 : b & 15) - z);
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (m0 + i < a.M)
                    for (int j = 0; j < n; ++j)
                        acc[i] = fmaf(w[j], to_float(x[(m0 + i) * a.x_stride + k + j]), acc[i]);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float t = acc[i];
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
            if (lane == 0 && m0 + i < a.M)
                y[(m0 + i) * a.y_stride + v] = from_float<T>(t + (a.bias ? a.bias[v] : 0.f));
        }
    }
}

struct QuantArgs {
    const void *w;
    int64_t V, K, w_stride;
    int group, symmetric;
    uint8_t *q;
    int64_t q_pitch;
    void *scales;
    int scale_dtype;
    int64_t s_stride;
    uint8_t *zeros;
    int64_t z_stride;
};

// One warp per group: its range, the scale as it will be stored, then the
// nibbles rounded against that stored scale.
template <typename T> __global__ void __launch_bounds__(256) k_quantize(QuantArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t G = (a.K + a.group - 1) / a.group, items = a.V * G;
    const T *w = (const T *)a.w;
    for (int64_t it = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; it < items;
         it += (int64_t)gridDim.x * (blockDim.x / 32)) {
        const int64_t v = it / G, g = it % G, k0 = g * a.group;
        const int n = a.K - k0 < a.group ? (int)(a.K - k0) : a.group;
        float lo = 0.f, hi = 0.f;
        bool bad = false;
        for (int j = lane; j < n; j += 32) {
            const float t = to_float(w[v * a.w_stride + k0 + j]);
            bad |= !(fabsf(t) <= 3.402823466e38f);
            lo = fminf(lo, t);
            hi = fmaxf(hi, t);
        }
        for (int o = 16; o; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
        }
        bad = __any_sync(~0u, bad);
        float s = a.symmetric ? fmaxf(lo / -8.f, hi / 7.f) : hi / 15.f - lo / 15.f;
        if (bad) s = __int_as_float(0x7fc00000);
        if (a.scale_dtype == CK_BF16) s = __bfloat162float(__float2bfloat16_rn(s));
        if (a.scale_dtype == CK_F16) s = __half2float(__float2half_rn(s));
        const float z = a.symmetric ? 8.f
                                    : s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
        if (lane == 0) {
            if (a.scale_dtype == CK_F32) ((float *)a.scales)[v * a.s_stride + g] = s;
            if (a.scale_dtype == CK_BF16)
                ((__nv_bfloat16 *)a.scales)[v * a.s_stride + g] = __float2bfloat16_rn(s);
            if (a.scale_dtype == CK_F16) ((__half *)a.scales)[v * a.s_stride + g] = __float2half_rn(s);
            if (!a.symmetric) a.zeros[v * a.z_stride + g] = (uint8_t)z;
        }
        for (int j = 2 * lane; j < n; j += 64) {
            uint32_t b = 0;
            for (int h = 0; h < 2; ++h) {
                float t = z;
                if (j + h < n && s > 0.f)
                    t = fminf(fmaxf(rintf(to_float(w[v * a.w_stride + k0 + j + h]) / s) + z, 0.f), 15.f);
                b |= (uint32_t)t << (4 * h);
            }
            a.q[v * a.q_pitch + (k0 + j) / 2] = (uint8_t)b;
        }
    }
}

bool known_group(int64_t g) { return g == 32 || g == 64 || g == 128; }

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_int4_matvec(const void *x, int64_t dtype, int64_t M, int64_t K,
                                    int64_t x_stride, const uint8_t *qweight, int64_t V,
                                    int64_t q_pitch, const void *scales, int64_t scale_dtype,
                                    int64_t s_stride, const uint8_t *zeros, int64_t z_stride,
                                    const float *bias, int64_t group, void *y, int64_t y_stride,
                                    void *stream) {
    if (!known_dtype(dtype) || !known_dtype(scale_dtype))
        return fail(CK_ERR_INVALID_ARG, "int4_matvec: unknown dtype");
    if (!known_group(group))
        return fail(CK_ERR_INVALID_ARG, "int4_matvec: group must be 32, 64 or 128, not %lld", (long long)group);
    if (M < 0 || K < 1 || V < 0) return fail(CK_ERR_INVALID_ARG, "int4_matvec: M, V >= 0 and K >= 1");
    if (K >= ((int64_t)1 << 30) || V >= ((int64_t)1 << 30) || M >= ((int64_t)1 << 30))
        return fail(CK_ERR_UNSUPPORTED, "int4_matvec: a size of 2^30 or more");
    if (M == 0 || V == 0) return CK_OK;
    if (!x || !qweight || !scales || !y) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (q_pitch % 16 != 0 || ((uintptr_t)qweight & 15u) != 0 || q_pitch < (K + 1) / 2)
        return fail(CK_ERR_INVALID_ARG,
                    "int4_matvec: weight rows must start at multiples of 16 bytes and hold (K + 1) / 2 bytes");
    if (s_stride < (K + group - 1) / group || (zeros && z_stride < (K + group - 1) / group) ||
        x_stride < 0 || y_stride < V)
        return fail(CK_ERR_INVALID_ARG, "int4_matvec: a row stride is shorter than its row");
    MatvecArgs a{x, M, K, x_stride, qweight, V, q_pitch, scales, (int)scale_dtype, s_stride, zeros,
                 z_stride, bias, (int)group, y, y_stride};
    const int64_t my = (M + kRows - 1) / kRows;
    const dim3 grid((unsigned)((V + 7) / 8), (unsigned)(my < 1024 ? my : 1024));
    with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        k_matvec<T><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    });
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_matvec launch");
}

extern "C" ck_status ck_int4_quantize(const void *w, int64_t dtype, int64_t V, int64_t K,
                                      int64_t w_stride, int64_t group, int64_t symmetric,
                                      uint8_t *qweight, int64_t q_pitch, void *scales,
                                      int64_t scale_dtype, int64_t s_stride, uint8_t *zeros,
                                      int64_t z_stride, void *stream) {
    if (!known_dtype(dtype) || !known_dtype(scale_dtype))
        return fail(CK_ERR_INVALID_ARG, "int4_quantize: unknown dtype");
    if (!known_group(group))
        return fail(CK_ERR_INVALID_ARG, "int4_quantize: group must be 32, 64 or 128, not %lld", (long long)group);
    if (V < 0 || K < 1) return fail(CK_ERR_INVALID_ARG, "int4_quantize: V >= 0 and K >= 1");
    if (K >= ((int64_t)1 << 30) || V >= ((int64_t)1 << 30))
        return fail(CK_ERR_UNSUPPORTED, "int4_quantize: a size of 2^30 or more");
    if (V == 0) return CK_OK;
    if (!w || !qweight || !scales || (!symmetric && !zeros))
        return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    const int64_t G = (K + group - 1) / group;
    if (q_pitch < (K + 1) / 2 || s_stride < G || (!symmetric && z_stride < G) || w_stride < 0)
        return fail(CK_ERR_INVALID_ARG, "int4_quantize: a row stride is shorter than its row");
    QuantArgs a{w, V, K, w_stride, (int)group, symmetric != 0, qweight, q_pitch, scales,
                (int)scale_dtype, s_stride, zeros, z_stride};
    const int64_t want = (V * G + 7) / 8, most = 16 * (int64_t)device_sms();
    const int grid = (int)(want < most ? want : most);
    with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        k_quantize<T><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
    });
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_quantize launch");
}
