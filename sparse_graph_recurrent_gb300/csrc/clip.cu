// ck_grad_norm, ck_clip_gradients: the root of the sum of squares over many tensors, and
// the tensors scaled so that it is at most a given one.
//
//   norm = sqrt(sum g^2), factor = min(1, max_norm / (norm + 1e-6)), out = g factor
//
// The tensors are cut into chunks of kChunkBytes, numbered through, and every CTA takes a
// run of them.  The first kernel leaves a sum for each CTA; the second, launched so that it
// takes its places while the first ends, adds up the CTAs' sums (each CTA for itself, in one
// order, so that results repeat) and scales its run from the end, where memory read last is
// still in L2.
//
// The list of tensors is an argument of the kernels: nothing is copied, and a captured
// call holds it.
//
// Squares leave the range of 32 bits long before numbers do.  Where a CTA's sum says that they
// have, it adds up its run again with numbers scaled by a power of 2; the sums of CTAs are
// of 64 bits.
//
// What bounds both is memory: the gradients are read twice and written once, except what L2
// holds from the first time.  207 MB out of place: 36 us for the norm (5.8 TB/s) and 64 for the
// scaling (6.4 TB/s).  Operations of 64 bits are slow here (a warp's takes an SM some 20
// cycles); with one for every thread, three sums and their reductions, they took 11 and 18 us
// of the two kernels, so one warp of a CTA does the few that there are.
#include <algorithm>
#include <vector>

#include "ck_types.h"

namespace ck {
namespace {

constexpr int kClipThreads = 256, kClipVecs = 4;
constexpr int kChunkBytes = kClipThreads * kClipVecs * 16;
constexpr int kFew = 32, kMany = 1000;  // tensors of a launch: the arguments then take 1 and 29 KB
constexpr int kClipCtas = 4;            // CTAs an SM
// What the second kernel finds in L2 of what the first has read, where that marks the rest as
// not to be held (79 M numbers, 207 MB: 100.4 us, 105.2 with all marked, 103.2 with none).
constexpr int kHeldBytes = 80 << 20;

template <int MOST> struct ClipList {
    const void *in[MOST];
    void *out[MOST];
    int64_t n[MOST];
    int32_t start[MOST + 1];  // the tensor's first chunk
    uint8_t dtype[MOST];
    int count;
    double *sums;    // [CTAs of all launches]
    int first;       // the CTAs of the launches before
    int all;         // of all launches
    float *norm;
    double max_norm;
    int held;        // chunks that the second kernel finds in L2
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Where chunk c lies: the tensor, and elements [lo, hi) of it.  Chunks begin at multiples of
// 16 bytes in memory; what lies before the first such place belongs to the first chunk.
struct Where {
    int i, vecs;         // pieces of 16 bytes, from element `body` on
    int64_t lo, body, hi;
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
    const int shift = a.dtype[lo] == CK_F32 ? 2 : 1;  // bytes of an element, as a power of 2
    const int64_t k = c - a.start[lo], n = a.n[lo];
    int head = (int)((16 - ((uintptr_t)a.in[lo] & 15)) & 15) >> shift;
    if (head > n) head = (int)n;
    w.body = head + k * (kChunkBytes >> shift);
    w.lo = k ? w.body : 0;
    w.hi = head + (k + 1) * (kChunkBytes >> shift);
    if (w.hi > n) w.hi = n;
    w.vecs = (int)((w.hi - w.body) >> (4 - shift));
    return w;
}

// This thread's pieces of a chunk, kClipVecs of them or fewer.
// last: nothing reads them after this, soon enough to find them in L2.
template <typename L> __device__ __forceinline__ void chunk_load(const L &a, const Where &w, bool last, uint4 (&v)[kClipVecs]) {
    const uint4 *p = (const uint4 *)((const char *)a.in[w.i] + (w.body << (a.dtype[w.i] == CK_F32 ? 2 : 1))) + threadIdx.x;
    if (last && w.vecs == kClipThreads * kClipVecs) {
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) v[j] = load_once(p + j * kClipThreads);
    } else if (w.vecs == kClipThreads * kClipVecs) {
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) v[j] = p[j * kClipThreads];
    } else {
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if ((int)threadIdx.x + j * kClipThreads < w.vecs) v[j] = p[j * kClipThreads];
        }
    }
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

// The sum of this thread's squares in a chunk; bits: those that any of its numbers has.
template <typename T> __device__ __forceinline__ float chunk_sum(const T *in, const Where &w, const uint4 (&v)[kClipVecs], uint32_t &bits) {
    constexpr int E = 16 / (int)sizeof(T);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        alignas(16) T t[E];
        memcpy(t, &v[j], 16);
        bits |= v[j].x | v[j].y | v[j].z | v[j].w;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(to_float(t[e]), to_float(t[e]), s);
    }
    const int64_t edge = w.lo + threadIdx.x, tail = w.body + w.vecs * E + threadIdx.x;
    if (edge < w.body) {
        bits |= to_float(in[edge]) != 0.f;
        s = fmaf(to_float(in[edge]), to_float(in[edge]), s);
    }
    if (tail < w.hi) {
        bits |= to_float(in[tail]) != 0.f;
        s = fmaf(to_float(in[tail]), to_float(in[tail]), s);
    }
    return s;
}

// The sum of the warps' numbers, in the first warp.  (A warp's operation of 64 bits takes some
// 20 cycles of its SM, so one warp adds them up: 13 of them, not 100.)
__device__ __forceinline__ double block_sum(double v, double *shared) {
    shared[threadIdx.x] = v;
    __syncthreads();
    double t = 0;
    if (threadIdx.x < 32) {
#pragma unroll
        for (int i = 0; i < kClipThreads / 32; ++i) t += shared[threadIdx.x + 32 * i];
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    return t;
}

__device__ __forceinline__ void run_of(int chunks, int &lo, int &hi) {
    lo = (int)((int64_t)chunks * blockIdx.x / gridDim.x);
    hi = (int)((int64_t)chunks * (blockIdx.x + 1) / gridDim.x);
}

// The same of a run's numbers each times a power of 2, in the first warp: for the few runs
// that need it, one by one.
template <int MOST> __device__ __noinline__ double scaled_sum(const ClipList<MOST> &a, int lo, int hi, float scale, double *shared) {
    float s = 0.f;
    double total = 0;
    for (int c = lo; c < hi; ++c) {
        const Where w = locate(a, c, 0);
        by_dtype(a.dtype[w.i], [&](auto *t) {
            const auto *in = (const std::remove_pointer_t<decltype(t)> *)a.in[w.i];
            float part = 0.f;
            for (int64_t e = w.lo + threadIdx.x; e < w.hi; e += kClipThreads) {
                const float g = to_float(in[e]) * scale;
                part = fmaf(g, g, part);
            }
            s += part;
        });
        if ((c - lo) % 32 == 31) total += s, s = 0.f;
    }
    __syncthreads();
    return block_sum(total + (double)s, shared) / ((double)scale * (double)scale);
}

template <int MOST>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) k_norm(const __grid_constant__ ClipList<MOST> a) {
    __shared__ double shared[kClipThreads];
    __shared__ double sum;
    pdl_wait();
    pdl_launch();  // only now: what the second kernel reads before it waits is there then
    int lo, hi;
    run_of(a.start[a.count], lo, hi);
    // what this run has in L2 at the end, if all do likewise
    const int keep = hi - (int)(a.held / gridDim.x);
    float part = 0.f;
    // a chunk ahead is under way while one is added up
    uint4 v[kClipVecs], next[kClipVecs];
    Where w{}, then{};
    if (hi > lo) {
        w = locate(a, lo, 0);
        chunk_load(a, w, lo < keep, v);
    }
    uint32_t bits = 0;
    double total = 0;
    for (int c = lo; c < hi; ++c) {
        if (c + 1 < hi) {
            then = locate(a, c + 1, w.i);
            chunk_load(a, then, c + 1 < keep, next);
        }
        by_dtype(a.dtype[w.i], [&](auto *t) { part += chunk_sum((const std::remove_pointer_t<decltype(t)> *)a.in[w.i], w, v, bits); });
        if ((c - lo) % 32 == 31) total += part, part = 0.f;
        w = then;
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) v[j] = next[j];
    }
    double s = block_sum(total + (double)part, shared);
    if (threadIdx.x == 0) sum = s;
    const bool some = __syncthreads_or(bits);
    // Squares that left 32 bits, or may have been lost below them beside what is left: once more,
    // of numbers made smaller, or larger.
    if (!(sum <= 3.402823466e38f))
        s = scaled_sum(a, lo, hi, 8.271806125530277e-25f, shared);  // 2^-80
    else if (sum < 8.67e-19 && some)  // 2^-60; not where all are 0
        s = scaled_sum(a, lo, hi, 1.8446744073709552e19f, shared);  // 2^64
    if (threadIdx.x == 0) a.sums[a.first + blockIdx.x] = s;
}

// The root of a number that is not negative, rounded to 32 bits: of its first 24 bits, and what
// the rest adds.  (The root of 64 bits takes some 30 of the slow operations.)
__device__ __forceinline__ float root(double s) {
    if (!(s > 0) || !(s <= 1.7976931348623157e308)) return (float)s;  // 0, infinite, NaN
    const long long bits = __double_as_longlong(s);
    const int half = ((int)(bits >> 52) - 1023) >> 1;                // (s is no subnormal: it is a square over 2^-298)
    const double m = __longlong_as_double(bits - ((long long)(2 * half) << 52));  // in [1, 4)
    const float y = sqrtf((float)m);
    return ldexpf(y + (float)(m - (double)y * (double)y) / (2.f * y), half);
}

// The norm from all CTAs' sums and what the gradients are multiplied with, in all threads.
struct Factor {
    float norm, by;
};
__device__ __forceinline__ Factor factor_of(const double *sums, int all, double max_norm) {
    __shared__ Factor f;
    if (threadIdx.x < 32) {
        double s = 0;
        for (int i = threadIdx.x; i < all; i += 32) s += load_l2(sums + i);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            f.norm = root(s);
            // max_norm / (norm + 1e-6), rounded once but for what a 32-bit quotient's rest loses
            const double d = (double)f.norm + 1e-6;
            if (max_norm >= d) {
                f.by = 1.f;
            } else if (f.norm > 3.402823466e38f) {
                f.by = 0.f;
            } else {  // (NaN stays; max_norm is below d, and so inside 32 bits)
                const float q = (float)max_norm / (float)d;
                f.by = q + (float)(max_norm - (double)q * d) / (float)d;
            }
        }
    }
    __syncthreads();
    return f;
}

template <int MOST> __global__ void __launch_bounds__(kClipThreads) k_norm_end(const __grid_constant__ ClipList<MOST> a) {
    pdl_wait();
    const Factor f = factor_of(a.sums, a.all, 0);
    if (threadIdx.x == 0) *a.norm = f.norm;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *in, T *out, const Where &w, uint4 (&v)[kClipVecs], float factor) {
    constexpr int E = 16 / (int)sizeof(T);
    const bool wide = ((uintptr_t)(out + w.body) & 15) == 0;
#pragma unroll
    for (int j = 0; j < kClipVecs; ++j) {
        if ((int)threadIdx.x + j * kClipThreads >= w.vecs) continue;
        alignas(16) T t[E];
        memcpy(t, &v[j], 16);
#pragma unroll
        for (int e = 0; e < E; ++e) t[e] = from_float<T>(to_float(t[e]) * factor);
        T *to = out + w.body + (threadIdx.x + j * kClipThreads) * E;
        if (wide) {
            memcpy(&v[j], t, 16);
            __stcs((uint4 *)to, v[j]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) to[e] = t[e];
        }
    }
    const int64_t head = w.lo + threadIdx.x, tail = w.body + w.vecs * E + threadIdx.x;
    if (head < w.body) out[head] = from_float<T>(to_float(in[head]) * factor);
    if (tail < w.hi) out[tail] = from_float<T>(to_float(in[tail]) * factor);
}

template <int MOST>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) k_clip(const __grid_constant__ ClipList<MOST> a) {
    int lo, hi;
    run_of(a.start[a.count], lo, hi);
    // a chunk ahead is under way while one is scaled
    uint4 v[kClipVecs], next[kClipVecs];
    Where w{}, then{};
    if (hi > lo) w = locate(a, hi - 1, 0);
    pdl_wait();
    if (hi > lo) chunk_load(a, w, true, v);
    const Factor all = factor_of(a.sums, a.all, a.max_norm);
    const float factor = all.by;
    if (blockIdx.x == 0 && a.first == 0 && threadIdx.x == 0) *a.norm = all.norm;
    for (int c = hi - 1; c >= lo; --c) {
        if (c > lo) {
            then = locate(a, c - 1, 0);
            if (factor != 1.f || a.in[then.i] != a.out[then.i]) chunk_load(a, then, true, next);
        }
        if (factor != 1.f || a.in[w.i] != a.out[w.i])
            by_dtype(a.dtype[w.i], [&](auto *t) {
                using T = std::remove_pointer_t<decltype(t)>;
                chunk_scale((const T *)a.in[w.i], (T *)a.out[w.i], w, v, factor);
            });
        w = then;
#pragma unroll
        for (int j = 0; j < kClipVecs; ++j) v[j] = next[j];
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

size_t clip_workspace(const ck_gradient *list, int64_t count) {
    // a sum for each CTA of a launch; a launch ends at kMany tensors or 2^31 chunks
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i)
        if (list[i].n) chunks += chunks_of(list[i]);
    const int64_t launches = 1 + count / kMany + chunks / ((int64_t)1 << 30);
    const int64_t most = launches * kClipCtas * device_sms();
    return (size_t)(chunks < most ? chunks : most) * sizeof(double);
}

struct Span {
    uintptr_t lo, hi;
    bool written;
};

bool by_begin(const Span &a, const Span &b) { return a.lo < b.lo; }

// Whether what one tensor writes is read or written for another.  A tensor clipped in its
// own place is one span.  What is written is looked at by itself first, by type: it often
// lies in the order of the list, one line of memory for a type, and what is read elsewhere.
bool tangled(const ck_gradient *list, int64_t count) {
    std::vector<Span> written[3], all;
    uintptr_t lo = UINTPTR_MAX, hi = 0, read_lo = UINTPTR_MAX, read_hi = 0;
    for (int64_t i = 0; i < count; ++i) {
        const ck_gradient &g = list[i];
        if (!g.n) continue;
        const uintptr_t bytes = (uintptr_t)g.n * dtype_size(g.dtype), to = (uintptr_t)g.out, from = (uintptr_t)g.grad;
        written[g.dtype].push_back({to, to + bytes, true});
        lo = std::min(lo, to), hi = std::max(hi, to + bytes);
        if (to != from) read_lo = std::min(read_lo, from), read_hi = std::max(read_hi, from + bytes);
    }
    for (std::vector<Span> &spans : written) {
        if (!std::is_sorted(spans.begin(), spans.end(), by_begin)) std::sort(spans.begin(), spans.end(), by_begin);
        const size_t before = all.size();
        all.insert(all.end(), spans.begin(), spans.end());
        if (before && before < all.size() && all[before].lo < all[before - 1].lo)
            std::inplace_merge(all.begin(), all.begin() + before, all.end(), by_begin);
    }
    // What is read: mostly far from the few stretches that are written
    std::vector<Span> stretches;
    for (const Span &s : all) {
        if (!stretches.empty() && s.lo <= stretches.back().hi + 4096)
            stretches.back().hi = std::max(stretches.back().hi, s.hi);
        else
            stretches.push_back(s);
    }
    bool near = read_lo < hi && read_hi > lo;  // (nothing read: false)
    if (near && stretches.size() <= 8) {
        near = false;
        for (int64_t i = 0; i < count && !near; ++i) {
            const ck_gradient &g = list[i];
            const uintptr_t from = (uintptr_t)g.grad, end = from + (uintptr_t)g.n * dtype_size(g.dtype);
            if (g.n && g.out != g.grad)
                for (const Span &s : stretches) near |= from < s.hi && end > s.lo;
        }
    }
    if (near) {
        const size_t before = all.size();
        for (int64_t i = 0; i < count; ++i) {
            const ck_gradient &g = list[i];
            const uintptr_t from = (uintptr_t)g.grad;
            if (g.n && g.out != g.grad) all.push_back({from, from + (uintptr_t)g.n * dtype_size(g.dtype), false});
        }
        std::sort(all.begin() + before, all.end(), by_begin);
        std::inplace_merge(all.begin(), all.begin() + before, all.end(), by_begin);
    }
    uintptr_t end_written = 0, end_read = 0;
    for (const Span &s : all) {
        if (s.lo < end_written || (s.written && s.lo < end_read)) return true;
        uintptr_t &end = s.written ? end_written : end_read;
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

// Fills a launch's list from entry `at` on; returns the entry that the next begins with, `count`
// where nothing but empty tensors is left.
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
    while (at < count && !list[at].n) ++at;
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
    a.held = kHeldBytes / kChunkBytes;
    cudaError_t e = cudaSuccess;
    int launches = 0;
    for (int64_t at = 0; at < count && e == cudaSuccess;) {
        at = fill(a, list, count, at);
        if (!a.count) break;
        const int grid = clip_grid(a.start[a.count]);
        e = launch_after(k_norm<MOST>, grid, a, true, s);
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
    // The first of the second kernels may start early: it waits before it reads what another has
    // written.  (With its first chunk read before that, 98 us of the largest case were 98 too.)
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
    const size_t need = clip_workspace(list, count);
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
    *bytes = clip_workspace(list, count);
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
