// ck_control_logits: penalties for repeated tokens, biases, grammar masks and
// temperature on a batch of logits, and in the same pass the next token.
#include <cooperative_groups.h>

#include "ck_philox.h"
#include "ck_types.h"

namespace cg = cooperative_groups;

namespace ck {
namespace {

constexpr int kLogitThreads = 512;
constexpr int kTile = 16384;  // most tokens whose counts one CTA holds at once
constexpr int kOct = 8;       // tokens a thread takes at a time

enum Pick { kNone, kGreedy, kSample };

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xff800000); }

// Scores in an order that unsigned integers have too; 0 for what is never
// picked (NaN, -inf).  The lower word prefers the lowest index.
__device__ __forceinline__ unsigned long long pick_key(float score, uint32_t v) {
    if (!(score > minus_inf())) return 0;
    const uint32_t b = __float_as_uint(score + 0.f);  // -0 counts as 0
    return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xFFFFFFFFu - v);
}
__device__ __forceinline__ float key_score(unsigned long long key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return key ? __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b) : minus_inf();
}

__device__ __forceinline__ float gumbel(uint32_t word) {
    // u in (0, 1): 2^-33 keeps it off 0, the minimum off 1
    const float u = fminf(__fadd_rn((float)word * 2.3283064365386963e-10f, 1.1641532182693481e-10f),
                          0.99999994f);
    return -logf(-log1pf(-u));
}

__device__ __forceinline__ int64_t row_len(const void *p, int64_t bits, int64_t b, int64_t L) {
    if (!p) return L;
    const int64_t n = bits == 32 ? (int64_t)((const int32_t *)p)[b] : ((const int64_t *)p)[b];
    return n < 0 ? 0 : n < L ? n : L;
}

// Controls of a row.
template <typename T> struct Row {
    const T *in;
    T *out;
    const float *bias;
    const uint32_t *mask;
    float rep, freq, pres, temp;

    __device__ __forceinline__ float penalised(float z, uint32_t c) const {
        z = z > 0.f ? z / rep : z * rep;
        return __fsub_rn(z, __fadd_rn(__fmul_rn((float)(c >> 1), freq), c > 1 ? pres : 0.f));
    }
    // Logit v after all controls, c what the table holds for it.
    __device__ __forceinline__ float at(int64_t v, uint32_t c) const {
        float z = to_float(in[v]);
        if (c) z = penalised(z, c);
        if (bias) z = __fadd_rn(z, bias[v]);
        if (mask && !(mask[v >> 5] >> (v & 31) & 1u)) z = minus_inf();
        return temp > 0.f ? z / temp : z;
    }
};

// count[v - t0] for the tokens t0 <= v < t1 of history[0 .. len): twice the number
// of occurrences from `prompt` on, odd or not zero where the token was seen at all.
// Additions of integers: their order does not matter.
template <typename I>
__device__ __forceinline__ void count_history(const I *h, int64_t len, int64_t prompt, int64_t t0, int64_t t1,
                                              uint32_t *count) {
    constexpr int kBatch = 8;
    for (int64_t i0 = threadIdx.x; i0 < len; i0 += kBatch * kLogitThreads) {
        I v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t i = i0 + k * kLogitThreads;
            v[k] = i < len ? h[i] : (I)-1;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t i = i0 + k * kLogitThreads;
            if ((int64_t)v[k] < t0 || (int64_t)v[k] >= t1) continue;
            if (i >= prompt)
                atomicAdd(&count[v[k] - t0], 2u);  // seen, and made here
            else
                atomicOr(&count[v[k] - t0], 1u);
        }
    }
}

// A cluster of CTAs takes one row, each a slice of the vocabulary; the row's best
// token meets in the first CTA's shared memory.  A thread takes eight tokens at a
// time, cut so that they are two blocks of the generator (sampling) or 16-byte pieces
// of the logits (else).
//
// What bounds it at large sizes is arithmetic: a token drawn costs a word of the
// generator and two logarithms.  The logarithms are spared: as -log1p(-u) >= u, the
// noise is at most -log u, which one approximate logarithm of a number no larger
// than u bounds from above; only tokens whose bound reaches the best score that
// their warp has seen are scored as defined, from the start.
template <typename T, int PICK>
__global__ void __launch_bounds__(kLogitThreads, 2) k_logits(const __grid_constant__ ck_logit_call a,
                                                         const __grid_constant__ PhiloxKeys keys) {
    extern __shared__ __align__(16) uint32_t count[];
    __shared__ unsigned long long best_cta, best_of[8];  // best_of: of the cluster's CTAs, in the first
    cg::cluster_group cluster = cg::this_cluster();
    const int64_t b = blockIdx.y;
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    if (PICK != kNone) {
        if (threadIdx.x == 0) best_cta = 0;
        __syncthreads();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    const int64_t per = ((a.V + ranks - 1) / ranks + 127) / 128 * 128;
    const int64_t s0 = rank * per, s1 = s0 + per < a.V ? s0 + per : a.V;
    Row<T> row;
    row.in = (const T *)a.logits + b * a.logits_stride;
    row.out = a.out ? (T *)a.out + b * a.out_stride : nullptr;
    row.bias = a.bias ? a.bias + b * a.bias_stride : nullptr;
    row.mask = a.mask ? (const uint32_t *)a.mask + b * a.mask_stride : nullptr;
    row.rep = a.repetition ? a.repetition[b] : a.repetition_all;
    row.freq = a.frequency ? a.frequency[b] : a.frequency_all;
    row.pres = a.presence ? a.presence[b] : a.presence_all;
    row.temp = a.temperature ? a.temperature[b] : a.temperature_all;
    const bool heat = row.temp > 0.f, noisy = PICK == kSample && heat;
    const float cool = heat ? 1.f / row.temp : 1.f;
    const int64_t len = a.history ? row_len(a.history_len, a.history_bits, b, a.L) : 0;
    const int64_t prompt = a.history && a.prompt_len ? row_len(a.prompt_len, a.history_bits, b, a.L) : 0;
    const int64_t e0 = b * a.V;
    const uint64_t step = PICK == kSample ? keys.at() : 0;
    // octs begin at tokens v with (v + cut) % 8 == 0
    const int cut = PICK == kSample ? (int)(e0 & 7) : (int)(((uintptr_t)row.in / sizeof(T)) & 7);
    const bool in_vec = (((uintptr_t)row.in - cut * sizeof(T)) & 15) == 0;
    const bool out_vec = (((uintptr_t)row.out - cut * sizeof(T)) & 15) == 0;
    const bool bias_vec = (((uintptr_t)row.bias - cut * sizeof(float)) & 15) == 0;
    unsigned long long best = 0;
    float floor = minus_inf();  // sampling: the best score that the warp has seen
    for (int64_t t0 = s0; t0 < s1; t0 += kTile) {
        const int64_t t1 = t0 + kTile < s1 ? t0 + kTile : s1;
        const int64_t q0 = (t0 + cut) / kOct, q1 = (t1 + cut + kOct - 1) / kOct;
        if (len > 0) {
            if (t0 > s0) __syncthreads();
            for (int i = threadIdx.x; i < (int)(q1 - q0) * 2; i += kLogitThreads)
                ((uint4 *)count)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            uint32_t *mine = count + cut;
            if (a.history_bits == 32)
                count_history((const int32_t *)a.history + b * a.history_stride, len, prompt, t0, t1, mine);
            else
                count_history((const int64_t *)a.history + b * a.history_stride, len, prompt, t0, t1, mine);
            __syncthreads();
        }
        for (int64_t qw = q0 + (threadIdx.x & ~31); qw < q1; qw += kLogitThreads) {
            const int64_t q = qw + (threadIdx.x & 31), v0 = q * kOct - cut;
            float z[kOct];
            uint32_t ok = 0;  // tokens that are there and allowed
            if (v0 >= t0 && v0 + kOct <= t1 && in_vec) {
                alignas(16) T t[kOct];
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                    ((uint4 *)t)[i] = __ldcs((const uint4 *)(row.in + v0) + i);
#pragma unroll
                for (int j = 0; j < kOct; ++j) z[j] = to_float(t[j]);
                ok = 0xff;
            } else {
#pragma unroll
                for (int j = 0; j < kOct; ++j) {
                    const bool in = v0 + j >= t0 && v0 + j < t1;
                    z[j] = in ? to_float(row.in[v0 + j]) : 0.f;
                    ok |= (uint32_t)in << j;
                }
            }
            const uint32_t there = ok;
            if (len > 0 && there) {
                const uint4 c0 = ((const uint4 *)count)[2 * (q - q0)], c1 = ((const uint4 *)count)[2 * (q - q0) + 1];
                if (c0.x | c0.y | c0.z | c0.w | c1.x | c1.y | c1.z | c1.w) {
                    const uint32_t c[kOct] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
                    for (int j = 0; j < kOct; ++j)
                        if (c[j]) z[j] = row.penalised(z[j], c[j]);
                }
            }
            if (row.bias) {
                if (there == 0xff && bias_vec) {
                    const float4 b0 = *(const float4 *)(row.bias + v0), b1 = *(const float4 *)(row.bias + v0 + 4);
                    const float bb[kOct] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
                    for (int j = 0; j < kOct; ++j) z[j] = __fadd_rn(z[j], bb[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < kOct; ++j)
                        if (there >> j & 1) z[j] = __fadd_rn(z[j], row.bias[v0 + j]);
                }
            }
            if (row.mask) {
                if (there == 0xff) {
                    const uint32_t *w = row.mask + (v0 >> 5);
                    const int from = (int)(v0 & 31);
                    ok = __funnelshift_r(w[0], from > 32 - kOct ? w[1] : 0u, from) & 0xff;
                } else {
#pragma unroll
                    for (int j = 0; j < kOct; ++j)
                        if ((there >> j & 1) && !(row.mask[(v0 + j) >> 5] >> ((v0 + j) & 31) & 1u)) ok &= ~(1u << j);
                }
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (!(ok >> j & 1)) z[j] = minus_inf();
            }
            if (heat) {
                // a product would do to find candidates, but is not what is returned
                if (PICK == kSample && !row.out) {
#pragma unroll
                    for (int j = 0; j < kOct; ++j) z[j] *= cool;
                } else if (row.temp != 1.f) {
#pragma unroll
                    for (int j = 0; j < kOct; ++j) z[j] = z[j] / row.temp;
                }
            }
            if (row.out) {
                if (there == 0xff && out_vec) {
                    alignas(16) T t[kOct];
#pragma unroll
                    for (int j = 0; j < kOct; ++j) t[j] = from_float<T>(z[j]);
#pragma unroll
                    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                        __stcs((uint4 *)(row.out + v0) + i, ((const uint4 *)t)[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < kOct; ++j)
                        if (there >> j & 1) row.out[v0 + j] = from_float<T>(z[j]);
                }
            }
            if constexpr (PICK != kNone) {
                if (!noisy) {
                    float top = minus_inf();
                    int at = 0;
#pragma unroll
                    for (int j = 0; j < kOct; ++j)
                        if (z[j] > top && (there >> j & 1)) top = z[j], at = j;  // of equal ones the first; no NaN
                    const unsigned long long k = pick_key(top, (uint32_t)(v0 + at));
                    best = k > best ? k : best;
                    continue;
                }
            }
            if constexpr (PICK == kSample) {
                uint4 r0, r1;
                philox_two((uint64_t)(e0 + v0) >> 2, step, keys, r0, r1);
                const uint32_t w[kOct] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
                // z + noise is at most this
                float high[kOct];
#pragma unroll
                for (int j = 0; j < kOct; ++j) {
                    const float u = __uint_as_float(0x3f800000u | w[j] >> 9) - 1.f;  // u or less
                    const float s = fmaf(__log2f(u), -0.6931472f, z[j]);
                    high[j] = there >> j & 1 ? fmaf(fabsf(s), 1e-6f, s) + 1e-4f : minus_inf();
                }
                for (;;) {
                    float top = minus_inf();
                    int at = -1;
#pragma unroll
                    for (int j = 0; j < kOct; ++j)
                        if (high[j] > top) top = high[j], at = j;
                    const bool may = at >= 0 && top >= floor;
                    if (!__any_sync(~0u, may)) break;
                    unsigned long long k = 0;
                    if (may) {
                        const int64_t v = v0 + at;
                        const uint32_t c = len > 0 ? count[cut + (v - t0)] : 0u;
                        const uint32_t word = at < 4 ? (at < 2 ? (at ? r0.y : r0.x) : (at < 3 ? r0.z : r0.w))
                                                     : (at < 6 ? (at < 5 ? r1.x : r1.y) : (at < 7 ? r1.z : r1.w));
                        // in place, the logit may be overwritten: z is then what is returned, in full
                        float zv = 0.f;
                        if (row.out) {
#pragma unroll
                            for (int j = 0; j < kOct; ++j)
                                if (j == at) zv = z[j];
                        } else {
                            zv = row.at(v, c);
                        }
                        k = pick_key(__fadd_rn(zv, gumbel(word)), (uint32_t)v);
                        best = k > best ? k : best;
#pragma unroll
                        for (int j = 0; j < kOct; ++j)
                            if (j == at) high[j] = minus_inf();
                    }
                    const uint32_t seen = __reduce_max_sync(~0u, (uint32_t)(k >> 32));
                    floor = fmaxf(floor, key_score((unsigned long long)seen << 32));
                }
            }
        }
    }
    if constexpr (PICK != kNone) {
        for (int o = 16; o; o >>= 1) {
            const unsigned long long k = __shfl_xor_sync(~0u, best, o);
            best = k > best ? k : best;
        }
        if ((threadIdx.x & 31) == 0 && best) atomicMax(&best_cta, best);
        __syncthreads();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the first CTA has begun
        if (threadIdx.x == 0) *cluster.map_shared_rank(&best_of[rank], 0) = best_cta;
        cluster.sync();
        if (rank == 0 && threadIdx.x == 0) {
            for (int i = 0; i < ranks; ++i) best = best_of[i] > best ? best_of[i] : best;
            a.tokens[b] = best ? (int64_t)(0xFFFFFFFFu - (uint32_t)best) : -1;
        }
    }
}

template <typename T, int PICK>
cudaError_t launch_logits(const ck_logit_call &a, const PhiloxKeys &keys, int ranks, size_t smem,
                          cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(k_logits<T, PICK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kTile + 2 * kOct) * (int)sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)a.B);
    cfg.blockDim = dim3(kLogitThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_logits<T, PICK>, a, keys);
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
    // A CTA for 4,096 tokens of a row, for 1,024 where rows are few; eight at most
    // make a cluster everywhere.
    const int64_t few = a.B * 8 < 4 * (int64_t)device_sms() ? 1024 : 4096;
    int ranks = 1;
    while (ranks < 8 && ranks * few < a.V) ranks *= 2;
    const int64_t per = ((a.V + ranks - 1) / ranks + 127) / 128 * 128;
    const size_t smem = a.history ? (size_t)((per < kTile ? per : kTile) + 2 * kOct) * sizeof(uint32_t) : 0;
    const PhiloxKeys keys = PhiloxKeys::of(a.seed, a.step, a.step_dev);
    cudaError_t e = cudaSuccess;
    with_dtype(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        cudaStream_t s = (cudaStream_t)stream;
        e = !a.tokens  ? launch_logits<T, kNone>(a, keys, ranks, smem, s)
            : a.sample ? launch_logits<T, kSample>(a, keys, ranks, smem, s)
                       : launch_logits<T, kGreedy>(a, keys, ranks, smem, s);
    });
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_logits launch");
}
