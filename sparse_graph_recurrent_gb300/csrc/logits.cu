// ck_control_logits: penalties for repeated tokens, biases, grammar masks and
// temperature on a batch of logits, and in the same pass the next token.
#include <cooperative_groups.h>

#include "ck_philox.h"
#include "ck_types.h"

namespace cg = cooperative_groups;

namespace ck {
namespace {

constexpr int kLogitThreads = 512;
constexpr int kTile = 8192;  // tokens whose counts one CTA holds at once

// Scores in an order that unsigned integers have too; 0 for what is never
// picked (NaN, -inf).  The lower word prefers the lowest index.
__device__ __forceinline__ uint64_t pick_key(float score, uint32_t v) {
    if (!(score > -__int_as_float(0x7f800000))) return 0;
    const uint32_t b = __float_as_uint(score + 0.f);  // -0 counts as 0
    return (uint64_t)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xFFFFFFFFu - v);
}

__device__ __forceinline__ float gumbel(uint32_t word) {
    // u in (0, 1): 2^-33 keeps it off 0, the minimum off 1
    const float u = fminf(__fadd_rn((float)word * 2.3283064365386963e-10f, 1.1641532182693481e-10f),
                          0.99999994f);
    return -logf(-log1pf(-u));
}

template <typename I> __device__ __forceinline__ int64_t row_len(const void *p, int64_t b, int64_t L) {
    if (!p) return L;
    const int64_t n = (int64_t)((const I *)p)[b];
    return n < 0 ? 0 : n < L ? n : L;
}

// A cluster of CTAs takes one row; each CTA a slice of the vocabulary, in
// tiles.  Counts of a tile's tokens are taken from the row's history with
// integer additions in shared memory, so their order does not matter.
template <typename T, typename I>
__global__ void __launch_bounds__(kLogitThreads) k_logits(const __grid_constant__ ck_logit_call a,
                                                         const __grid_constant__ PhiloxKeys keys) {
    __shared__ uint32_t count[kTile];
    __shared__ uint64_t best_of[32];
    __shared__ uint64_t best_cta;
    cg::cluster_group cluster = cg::this_cluster();
    const int64_t b = blockIdx.y;
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int64_t per = ((a.V + ranks - 1) / ranks + 127) / 128 * 128;
    const int64_t s0 = rank * per, s1 = s0 + per < a.V ? s0 + per : a.V;
    const uint64_t step = keys.at();
    const float rep = a.repetition ? a.repetition[b] : a.repetition_all;
    const float freq = a.frequency ? a.frequency[b] : a.frequency_all;
    const float pres = a.presence ? a.presence[b] : a.presence_all;
    const float temp = a.temperature ? a.temperature[b] : a.temperature_all;
    const bool heat = temp > 0.f, noisy = a.sample && heat;
    const int64_t len = a.history ? row_len<I>(a.history_len, b, a.L) : 0;
    const int64_t prompt = a.history && a.prompt_len ? row_len<I>(a.prompt_len, b, a.L) : 0;
    const I *hist = (const I *)a.history + b * a.history_stride;
    const T *in = (const T *)a.logits + b * a.logits_stride;
    T *out = a.out ? (T *)a.out + b * a.out_stride : nullptr;
    const float *bias = a.bias ? a.bias + b * a.bias_stride : nullptr;
    const uint32_t *mask = a.mask ? (const uint32_t *)a.mask + b * a.mask_stride : nullptr;
    uint64_t best = 0;
    for (int64_t t0 = s0; t0 < s1; t0 += kTile) {
        const int64_t t1 = t0 + kTile < s1 ? t0 + kTile : s1;
        if (len > 0) {
            for (int i = threadIdx.x; i < kTile; i += kLogitThreads) count[i] = 0;
            __syncthreads();
            for (int64_t i = threadIdx.x; i < len; i += kLogitThreads) {
                const int64_t v = (int64_t)hist[i];
                if (v < t0 || v >= t1) continue;
                if (i >= prompt)
                    atomicAdd(&count[v - t0], 2u);  // seen, and made here
                else
                    atomicOr(&count[v - t0], 1u);
            }
            __syncthreads();
        }
        // quads of the generator's elements b V + v, so that a word is made once
        const int64_t e0 = b * a.V;
        for (int64_t q = (e0 + t0) / 4 + threadIdx.x; 4 * q < e0 + t1; q += kLogitThreads) {
            uint4 r = make_uint4(0, 0, 0, 0);
            if (noisy) r = philox((uint64_t)q, step, keys);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t v = 4 * q + j - e0;
                if (v < t0 || v >= t1) continue;
                float z = to_float(in[v]);
                const uint32_t c = len > 0 ? count[v - t0] : 0u;
                if (c) {
                    z = z > 0.f ? z / rep : z * rep;
                    z = __fsub_rn(z, __fadd_rn(__fmul_rn((float)(c >> 1), freq), c > 1 ? pres : 0.f));
                }
                if (bias) z = __fadd_rn(z, bias[v]);
                if (mask && !(mask[v >> 5] >> (v & 31) & 1u)) z = -__int_as_float(0x7f800000);
                if (heat) z = z / temp;
                if (out) out[v] = from_float<T>(z);
                if (a.tokens) {
                    const uint64_t k = pick_key(noisy ? __fadd_rn(z, gumbel(w[j])) : z, (uint32_t)v);
                    best = k > best ? k : best;
                }
            }
        }
        __syncthreads();
    }
    if (!a.tokens) return;
    for (int o = 16; o; o >>= 1) {
        const uint64_t k = __shfl_xor_sync(~0u, best, o);
        best = k > best ? k : best;
    }
    if ((threadIdx.x & 31) == 0) best_of[threadIdx.x / 32] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kLogitThreads / 32; ++i) best = best_of[i] > best ? best_of[i] : best;
        best_cta = best;
    }
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
        for (int i = 1; i < ranks; ++i) {
            const uint64_t k = *cluster.map_shared_rank(&best_cta, i);
            best = k > best ? k : best;
        }
        a.tokens[b] = best ? (int64_t)(0xFFFFFFFFu - (uint32_t)best) : -1;
    }
    cluster.sync();  // no CTA leaves while its shared memory is read
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_control_logits(const ck_logit_call *call, void *stream) {
    if (!call) return fail(CK_ERR_INVALID_ARG, "control_logits: call is NULL");
    const ck_logit_call &a = *call;
    if (!known_dtype(a.dtype)) return fail(CK_ERR_INVALID_ARG, "control_logits: unknown dtype");
    if (a.B < 0 || a.V < 1) return fail(CK_ERR_INVALID_ARG, "control_logits: B >= 0 and V >= 1");
    if (a.V >= ((int64_t)1 << 31) || a.B > 65535)
        return fail(CK_ERR_UNSUPPORTED, "control_logits: V < 2^31 and B <= 65535");
    if (a.B == 0) return CK_OK;
    if (!a.logits || (!a.out && !a.tokens)) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (a.history && ((a.history_bits != 32 && a.history_bits != 64) || a.L < 0 || a.L >= ((int64_t)1 << 30)))
        return fail(CK_ERR_INVALID_ARG, "control_logits: history of 32 or 64 bits, 0 <= L < 2^30");
    int64_t ranks = 1;
    while (ranks < 8 && ranks * 4096 < a.V) ranks *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)a.B);
    cfg.blockDim = dim3(kLogitThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const PhiloxKeys keys = PhiloxKeys::of(a.seed, a.step, a.step_dev);
    cudaError_t e = cudaSuccess;
    with_dtype(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        e = a.history && a.history_bits == 32 ? cudaLaunchKernelEx(&cfg, k_logits<T, int32_t>, a, keys)
                                              : cudaLaunchKernelEx(&cfg, k_logits<T, int64_t>, a, keys);
    });
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_logits launch");
}
