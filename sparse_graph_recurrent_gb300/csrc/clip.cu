// ck_grad_norm, ck_clip_gradients: the root of the sum of squares over many tensors, and
// the tensors scaled so that it is at most a given one.
//
//   norm = sqrt(sum g^2), factor = min(1, max_norm / (norm + 1e-6)), out = g factor
//
// The tensors are cut into chunks of kChunkBytes, numbered through, and every CTA takes a
// run of them.  The first kernel leaves a sum for each CTA; the second, launched so that it
// starts while the first ends, reads its first chunk, adds up the CTAs' sums (each CTA for
// itself, in one order, so that results repeat) and scales its run from the end, where
// memory read last is still in L2.
//
// The list of tensors is an argument of the kernels: nothing is copied, and a captured
// call holds it.
//
// Squares leave the range of 32 bits long before numbers do.  So three sums are kept: of
// g^2, of (g 2^-80)^2 for when that overflows and of (g 2^64)^2 for when it is so small
// that squares were lost.
//
// What bounds both is memory: the gradients are read twice and written once, except what L2
// holds from the first time.
#include <algorithm>
#include <vector>

#include "ck_types.h"

namespace ck {
namespace {

constexpr int kClipThreads = 256, kClipVecs = 4;
constexpr int kChunkBytes = kClipThreads * kClipVecs * 16;
constexpr int kFew = 32, kMany = 1000;  // tensors of a launch: the arguments then take 1 and 29 KB
constexpr int kClipCtas = 4;            // CTAs an SM

struct Sums {
    float mid, big, small;
};

template <int MOST> struct ClipList {
    const void *in[MOST];
    void *out[MOST];
    int64_t n[MOST];
    int32_t start[MOST + 1];  // the tensor's first chunk
    uint8_t dtype[MOST];
    int count;
    double *sums;    // [CTAs of all launches][3]
    int first;       // the CTAs of the launches before
    int all;         // of all launches
    float *norm;
    double max_norm;
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Where chunk c lies: the tensor, and elements [lo, hi) of it.  Chunks begin at multiples of
// 16 bytes in memory; what lies before the first such place belongs to the first chunk.
struct Where {
    int i;
    int64_t lo, hi;
    int head;  // elements before the first multiple of 16 bytes
};

template <typename L> __device__ __forceinline__ Where locate(const L &a, int c, int from) {
    int lo = from, hi = a.count - 1;
    while (lo < hi) {  // the last tensor that starts at or before c
        const int m = (lo + hi + 1) / 2;
        if (a.start[m] <= c)
            lo = m;
        else
            hi = m - 1;
    }
    Where w;
    w.i = lo;
    const int e = a.dtype[lo] == CK_F32 ? 4 : 2;
    const int64_t per = kChunkBytes / e, k = c - a.start[lo], n = a.n[lo];
    w.head = (int)((16 - ((uintptr_t)a.in[lo] & 15)) & 15) / e;
    if (w.head > n) w.head = (int)n;
    w.lo = k ? w.head + k * per : 0;
    w.hi = w.head + (k + 1) * per;
    if (w.hi > n) w.hi = n;
    return w;
}

template <typename T> struct Scaled {
    // Only where a type's squares may leave 32 bits.
    static constexpr bool kThree = !std::is_same<T, __half>::value;
};

template <typename T> __device__ __forceinline__ void add_square(Sums &s, T g) {
    const float v = to_float(g);
    s.mid = fmaf(v, v, s.mid);
    if constexpr (Scaled<T>::kThree) {
        const float b = v * 8.271806125530277e-25f, t = v * 1.8446744073709552e19f;
        s.big = fmaf(b, b, s.big);
        s.small = fmaf(t, t, s.small);
    }
}

template <typename T> __device__ __forceinline__ void chunk_sum(const T *in, const Where &w, Sums &total) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t body = w.lo > w.head ? w.lo : w.head;  // a multiple of 16 bytes in memory
    const int64_t vecs = (w.hi - body) / E;
    const uint4 *p = (const uint4 *)(in + body);
    uint4 v[kClipVecs];
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j)
        if (threadIdx.x + j * kClipThreads < vecs) v[j] = __ldg(p + threadIdx.x + j * kClipThreads);
    Sums s{0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        if (threadIdx.x + j * kClipThreads >= vecs) continue;
        alignas(16) T t[E];
        memcpy(t, &v[j], 16);
#pragma unroll
        for (int e = 0; e < E; ++e) add_square(s, t[e]);
    }
    if (w.lo + threadIdx.x < body) add_square(s, in[w.lo + threadIdx.x]);
    const int64_t tail = body + vecs * E + threadIdx.x;
    if (tail < w.hi) add_square(s, in[tail]);
    total.mid += s.mid;
    total.big += s.big;
    total.small += s.small;
    if constexpr (!Scaled<T>::kThree) {
        if (!(s.mid <= 3.402823466e38f)) total.big += s.mid;  // infinities and NaN
    }
}

__device__ __forceinline__ double block_sum(double v, double *shared) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0;
#pragma unroll
    for (int i = 0; i < kClipThreads / 32; ++i) t += shared[i];
    __syncthreads();
    return t;
}

__device__ __forceinline__ void run_of(int chunks, int &lo, int &hi) {
    lo = (int)((int64_t)chunks * blockIdx.x / gridDim.x);
    hi = (int)((int64_t)chunks * (blockIdx.x + 1) / gridDim.x);
}

template <int MOST> __global__ void __launch_bounds__(kClipThreads) k_norm(const __grid_constant__ ClipList<MOST> a) {
    __shared__ double shared[kClipThreads / 32];
    pdl_launch();
    int lo, hi, i = 0;
    run_of(a.start[a.count], lo, hi);
    Sums s{0.f, 0.f, 0.f};
    for (int c = lo; c < hi; ++c) {
        const Where w = locate(a, c, i);
        i = w.i;
        if (a.dtype[i] == CK_F32)
            chunk_sum((const float *)a.in[i], w, s);
        else if (a.dtype[i] == CK_BF16)
            chunk_sum((const __nv_bfloat16 *)a.in[i], w, s);
        else
            chunk_sum((const __half *)a.in[i], w, s);
    }
    const double mid = block_sum(s.mid, shared), big = block_sum(s.big, shared), small = block_sum(s.small, shared);
    if (threadIdx.x == 0) {
        double *to = a.sums + 3 * (a.first + blockIdx.x);
        to[0] = mid, to[1] = big, to[2] = small;
    }
}

// The norm from all CTAs' sums.
__device__ __forceinline__ float norm_of(const double *sums, int all, double *shared) {
    double mid = 0, big = 0, small = 0;
    for (int i = threadIdx.x; i < all; i += kClipThreads) {
        mid += __ldcg(sums + 3 * i);
        big += __ldcg(sums + 3 * i + 1);
        small += __ldcg(sums + 3 * i + 2);
    }
    mid = block_sum(mid, shared), big = block_sum(big, shared), small = block_sum(small, shared);
    if (!(mid <= 1.7976931348623157e308)) return (float)(sqrt(big) * 1.2089258196146292e24);  // 2^80; inf and NaN too
    if (mid < 8.67e-19) return (float)(sqrt(small) * 5.421010862427522e-20);                   // 2^-60, 2^-64
    return (float)sqrt(mid);
}

template <int MOST> __global__ void __launch_bounds__(kClipThreads) k_norm_end(const __grid_constant__ ClipList<MOST> a) {
    __shared__ double shared[kClipThreads / 32];
    pdl_wait();
    const float n = norm_of(a.sums, a.all, shared);
    if (threadIdx.x == 0) *a.norm = n;
}

template <typename T>
__device__ __forceinline__ void chunk_load(const T *in, const Where &w, uint4 (&v)[kClipVecs]) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t body = w.lo > w.head ? w.lo : w.head, vecs = (w.hi - body) / E;
    const uint4 *p = (const uint4 *)(in + body);
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j)
        if (threadIdx.x + j * kClipThreads < vecs) v[j] = p[threadIdx.x + j * kClipThreads];
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *in, T *out, const Where &w, uint4 (&v)[kClipVecs], float factor) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t body = w.lo > w.head ? w.lo : w.head, vecs = (w.hi - body) / E;
    const bool wide = ((uintptr_t)(out + body) & 15) == 0;
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        if (threadIdx.x + j * kClipThreads >= vecs) continue;
        alignas(16) T t[E];
        memcpy(t, &v[j], 16);
#pragma unroll
        for (int e = 0; e < E; ++e) t[e] = from_float<T>(to_float(t[e]) * factor);
        T *to = out + body + (threadIdx.x + j * kClipThreads) * E;
        if (wide) {
            memcpy(&v[j], t, 16);
            __stcs((uint4 *)to, v[j]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) to[e] = t[e];
        }
    }
    const int64_t head = w.lo + threadIdx.x, tail = body + vecs * E + threadIdx.x;
    if (head < body) out[head] = from_float<T>(to_float(in[head]) * factor);
    if (tail < w.hi) out[tail] = from_float<T>(to_float(in[tail]) * factor);
}

// f((T *)nullptr) with T the element type.
template <typename F> __device__ __forceinline__ void by_dtype(uint8_t d, F &&f) {
    if (d == CK_F32)
        f((float *)nullptr);
    else if (d == CK_BF16)
        f((__nv_bfloat16 *)nullptr);
    else
        f((__half *)nullptr);
}

template <int MOST> __global__ void __launch_bounds__(kClipThreads) k_clip(const __grid_constant__ ClipList<MOST> a) {
    __shared__ double shared[kClipThreads / 32];
    int lo, hi;
    run_of(a.start[a.count], lo, hi);
    uint4 v[kClipVecs];
    Where w{};
    auto load = [&]() {
        by_dtype(a.dtype[w.i], [&](auto *t) { chunk_load((const std::remove_pointer_t<decltype(t)> *)a.in[w.i], w, v); });
    };
    if (hi > lo) {
        w = locate(a, hi - 1, 0);
        load();
    }
    pdl_wait();
    const float norm = norm_of(a.sums, a.all, shared);
    const float f = (float)(a.max_norm / ((double)norm + 1e-6));
    const float factor = f >= 1.f ? 1.f : f;  // (NaN stays)
    if (blockIdx.x == 0 && a.first == 0 && threadIdx.x == 0) *a.norm = norm;
    for (int c = hi - 1; c >= lo; --c) {
        if (c < hi - 1) w = locate(a, c, 0);
        if (factor == 1.f && a.in[w.i] == a.out[w.i]) continue;
        if (c < hi - 1) load();
        by_dtype(a.dtype[w.i], [&](auto *t) {
            using T = std::remove_pointer_t<decltype(t)>;
            chunk_scale((const T *)a.in[w.i], (T *)a.out[w.i], w, v, factor);
        });
    }
}

int64_t chunks_of(const ck_gradient &g) {
    const int64_t e = (int64_t)dtype_size(g.dtype), head = (int64_t)((16 - ((uintptr_t)g.grad & 15)) & 15) / e;
    const int64_t per = kChunkBytes / e;
    return g.n <= head ? 1 : (g.n - head + per - 1) / per;
}

ck_status check_list(const ck_gradient *list, int64_t count, bool clip) {
    if (count < 0 || (count && !list)) return fail(CK_ERR_INVALID_ARG, "gradients: no list");
    for (int64_t i = 0; i < count; ++i) {
        const ck_gradient &g = list[i];
        if (!known_dtype(g.dtype)) return fail(CK_ERR_INVALID_ARG, "gradients: unknown dtype %lld", (long long)g.dtype);
        if (g.n < 0) return fail(CK_ERR_INVALID_ARG, "gradients: negative size");
        if (g.n > ((int64_t)1 << 40)) return fail(CK_ERR_UNSUPPORTED, "gradients: more than 2^40 elements");
        if (g.n && (!g.grad || (clip && !g.out))) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
        if (!aligned(g.grad, dtype_size(g.dtype)) || (clip && !aligned(g.out, dtype_size(g.dtype))))
            return fail(CK_ERR_INVALID_ARG, "gradients: a pointer is not aligned to its elements");
    }
    return CK_OK;
}

struct Span {
    uintptr_t lo, hi;
    bool written;
};

// Whether what one tensor writes is read or written for another.  A tensor clipped in its
// own place is one span.
bool tangled(const ck_gradient *list, int64_t count) {
    std::vector<Span> spans;
    spans.reserve(2 * (size_t)count);
    for (int64_t i = 0; i < count; ++i) {
        const ck_gradient &g = list[i];
        if (!g.n) continue;
        const uintptr_t bytes = (uintptr_t)g.n * dtype_size(g.dtype);
        spans.push_back({(uintptr_t)g.out, (uintptr_t)g.out + bytes, true});
        if (g.out != g.grad) spans.push_back({(uintptr_t)g.grad, (uintptr_t)g.grad + bytes, false});
    }
    const auto before = [](const Span &a, const Span &b) { return a.lo < b.lo; };
    if (!std::is_sorted(spans.begin(), spans.end(), before)) std::sort(spans.begin(), spans.end(), before);
    uintptr_t written = 0, read = 0;
    for (const Span &s : spans) {
        if (s.lo < written || (s.written && s.lo < read)) return true;
        uintptr_t &end = s.written ? written : read;
        end = std::max(end, s.hi);
    }
    return false;
}

template <typename K, typename A> cudaError_t launch_after(K kernel, int grid, const A &a, bool early, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kClipThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Fills a launch's list from entry `at` on; returns the entry after its last.
template <int MOST> int64_t fill(ClipList<MOST> &a, const ck_gradient *list, int64_t count, int64_t at) {
    a.count = 0;
    int64_t chunks = 0;
    for (; at < count && a.count < MOST; ++at) {
        const ck_gradient &g = list[at];
        if (!g.n) continue;
        const int64_t c = chunks_of(g);
        if (chunks + c > 0x7fffffff) break;
        a.in[a.count] = g.grad;
        a.out[a.count] = g.out;
        a.n[a.count] = g.n;
        a.dtype[a.count] = (uint8_t)g.dtype;
        a.start[a.count++] = (int32_t)chunks;
        chunks += c;
    }
    a.start[a.count] = (int32_t)chunks;
    return at;
}

int clip_grid(int chunks) {
    const int most = kClipCtas * device_sms();
    return chunks < most ? chunks : most;
}

template <int MOST>
ck_status run_clip(const ck_gradient *list, int64_t count, bool clip, double max_norm, float *norm, double *sums,
                   cudaStream_t s) {
    ClipList<MOST> a;
    a.sums = sums;
    a.norm = norm;
    a.max_norm = max_norm;
    a.all = a.first = 0;
    cudaError_t e = cudaSuccess;
    int launches = 0;
    for (int64_t at = 0; at < count && e == cudaSuccess;) {
        at = fill(a, list, count, at);
        if (!a.count) break;
        const int grid = clip_grid(a.start[a.count]);
        k_norm<MOST><<<grid, kClipThreads, 0, s>>>(a);
        e = cudaGetLastError();
        a.first += grid;
        ++launches;
    }
    a.all = a.first;
    a.first = 0;
    if (e != cudaSuccess) return cuda_fail(e, "k_norm launch");
    if (!clip || !launches) {
        e = launch_after(k_norm_end<MOST>, 1, a, launches > 0, s);
        return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_norm_end launch");
    }
    // The first of the second kernels may start early: all it reads before it waits are
    // gradients, which no kernel of this call has written yet.
    bool early = true;
    for (int64_t at = 0; at < count && e == cudaSuccess;) {
        if (launches > 1) at = fill(a, list, count, at);
        else at = count;
        if (!a.count) break;
        const int grid = clip_grid(a.start[a.count]);
        e = launch_after(k_clip<MOST>, grid, a, early, s);
        early = false;
        a.first += grid;
    }
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_clip launch");
}

ck_status clip_call(const ck_gradient *list, int64_t count, bool clip, double max_norm, float *norm, void *workspace,
                    int64_t workspace_bytes, void *stream) {
    ck_status st = check_list(list, count, clip);
    if (st != CK_OK) return st;
    if (!norm) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (clip && !(max_norm >= 0)) return fail(CK_ERR_INVALID_ARG, "gradients: max_norm must be a number of at least 0");
    if (!aligned(norm, 4) || !aligned(workspace, 8))
        return fail(CK_ERR_INVALID_ARG, "gradients: a pointer is not aligned to its elements");
    size_t need = 0;
    st = ck_clip_workspace_size(list, count, &need);
    if (st != CK_OK) return st;
    if (need && (!workspace || (size_t)workspace_bytes < need))
        return fail(CK_ERR_WORKSPACE, "gradients: a workspace of %zu bytes is needed", need);
    if (clip) {
        try {
            if (tangled(list, count)) return fail(CK_ERR_INVALID_ARG, "gradients: two tensors share memory that is written");
        } catch (const std::exception &) {
            return fail(CK_ERR_OUT_OF_MEMORY, "gradients: no host memory for %lld tensors", (long long)count);
        }
    }
    const cudaStream_t s = (cudaStream_t)stream;
    return count <= kFew ? run_clip<kFew>(list, count, clip, max_norm, norm, (double *)workspace, s)
                         : run_clip<kMany>(list, count, clip, max_norm, norm, (double *)workspace, s);
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_clip_workspace_size(const ck_gradient *list, int64_t count, size_t *bytes) {
    const ck_status st = check_list(list, count, false);
    if (st != CK_OK) return st;
    if (!bytes) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    // three sums for each CTA of a launch; a launch ends at kMany tensors or 2^31 chunks
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i)
        if (list[i].n) chunks += chunks_of(list[i]);
    const int64_t launches = 1 + count / kMany + chunks / ((int64_t)1 << 30);
    const int64_t most = launches * kClipCtas * device_sms();
    *bytes = (size_t)(chunks < most ? chunks : most) * 3 * sizeof(double);
    return CK_OK;
}

extern "C" ck_status ck_grad_norm(const ck_gradient *list, int64_t count, float *norm, void *workspace,
                                  int64_t workspace_bytes, void *stream) {
    return clip_call(list, count, false, 0, norm, workspace, workspace_bytes, stream);
}

extern "C" ck_status ck_clip_gradients(const ck_gradient *list, int64_t count, double max_norm, float *norm,
                                       void *workspace, int64_t workspace_bytes, void *stream) {
    return clip_call(list, count, true, max_norm, norm, workspace, workspace_bytes, stream);
}
