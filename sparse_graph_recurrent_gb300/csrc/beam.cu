// ck_beam_select: of a beam search's K V candidates for each sequence the best, and
// ck_reorder_states: the beams' states moved to the places of those that were kept.
//
// The selection reads the logits once.  A CTA takes a slice of a beam's row into registers
// and leaves the slice's maximum, its sum of exponentials and its best candidates: the
// score's other terms are the same for all of a row, so inside one the order is that of
// the logits.  A second kernel, a CTA for each sequence, joins the slices' sums and picks
// from their lists.  Scores are added up and compared in 64 bits, but a row's sum is one of
// 32-bit exponentials, 32 in a row added in 32 bits, and so is its logarithm but for what its
// argument lost: there are few units for 64 bits.  It is off by (36 + 1.2 (ln V + 1)) 2^-23 at most.
//
// Both select alike.  The threads are put into 32 groups, one for each lane, and the groups'
// maxima are numbers of which the `beams`-th largest bounds the `beams`-th best from below,
// as so many are at least that.  What reaches the bound is gathered (with 16 beams and
// logits in no order some 22 of a slice) and ranked by counting.  Where that is too much (many
// equal ones, or all of the best in few groups' hands), or there are more beams than groups,
// the bound is found again from all threads' maxima, one after another and equal ones told
// apart by their tokens.
//
// What bounds it: of 16 x 16 beams over 131,072 bf16 logits the first kernel takes 18 us, 10 of
// them what memory needs; instructions (12 for a logit, 5 of them its exponential) and the
// waiting of a CTA's warps for one another are the rest.  The second takes 5, a chain of
// latencies.  Small calls are bound by the host.
#include <algorithm>
#include <vector>

#include "ck_types.h"

namespace ck {
namespace {

constexpr int kBeamThreads = 256, kBeamWarps = kBeamThreads / 32;
// 16-byte pieces of a thread (16 x 16 beams over 131,072 bf16 logits and their states: 35 us; with
// slices of 16, 48 and 64 KB instead of 32 41, 37 and 37)
constexpr int kBeamVecs = 8;
template <typename T> constexpr int kSlice = kBeamThreads * kBeamVecs * 16 / (int)sizeof(T);  // elements of a slice
inline int64_t slice_of(int64_t dtype) { return kBeamThreads * kBeamVecs * 16 / (int64_t)dtype_size(dtype); }
constexpr int kFound = 4096;  // 64 beams' threads' elements
constexpr int kAhead = 2;     // candidates that a thread of the second kernel asks for at once
constexpr int kFew = 512;     // more than this are not ranked without looking for a closer bound
constexpr int kMostBeams = 64;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ void beam_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void beam_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct BeamArgs {
    const void *logits;
    int64_t K, V, row, beam;
    const float *scores;
    const uint8_t *ended;
    int64_t end_token;
    int beams, slices;
    float *scores_out;
    int64_t *parents, *tokens;
    uint8_t *ended_out;
    // workspace, by slice: [B][K][slices], and [beams] candidates of each, best first
    double *sum;
    float *top;
    int *count;
    float *value;
    int *token;
};

// Floats in the order of unsigned integers; -inf is the lowest that occurs.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(uint64_t u) {
    return __longlong_as_double((long long)(u >> 63 ? u & 0x7fffffffffffffffull : ~u));
}

// Whether beam k of sequence b goes on by its logits.
__device__ __forceinline__ bool alive(const BeamArgs &a, int64_t at) {
    const float s = a.scores[at];
    return fabsf(s) <= 3.402823466e38f && !(a.ended && a.ended[at]);
}

// 2^x to 2 units; 0 below 2^-126.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float power(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// log(v) of a normal number above 0, to some 3e-8: there are few units for 64 bits, and v is no
// more exact than that.  v = 2^k m with m in [0.75, 1.5), m as a 32-bit float and what that lost.
__device__ __forceinline__ double log_of_sum(double v) {
    const long long bits = __double_as_longlong(v);
    int k = (int)(bits >> 52) - 1023;
    double m = __longlong_as_double((bits & 0xfffffffffffffll) | 0x3ff0000000000000ll);
    if (m >= 1.5) m *= 0.5, ++k;
    const float f = (float)m, lost = (float)(m - (double)f);
    return (double)k * 0.6931471805599453 + (double)(logf(f) + lost / f);
}

// The k-th largest (k <= 32) of the lanes' numbers, but for their last 5 bits (those are 0).
// Lanes with nothing have less than 32.
__device__ __forceinline__ uint32_t kth_of_warp(uint32_t mine, int k) {
    const int lane = threadIdx.x & 31;
    mine = mine < 32 ? lane : (mine & ~31u) | lane;  // all different
    int larger = 0;
#pragma unroll
    for (int o = 1; o < 32; ++o) larger += __shfl_sync(0xffffffffu, mine, lane + o) > mine;
    const uint32_t at = __ballot_sync(0xffffffffu, larger == k - 1);
    return __shfl_sync(0xffffffffu, mine, __ffs(at) - 1) & ~31u;
}

// Two elements of a piece of 16 bytes, NaN made -inf, and their larger one.
template <typename T> struct Pieces;
template <> struct Pieces<float> {
    static constexpr int E = 4;
    static constexpr uint32_t kNothing = 0xff800000u;
    static __device__ __forceinline__ uint32_t clean(uint32_t w) { return __float_as_uint(fmaxf(__uint_as_float(w), neg_inf())); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float one(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t bound(float z) { return __float_as_uint(z); }
    static __device__ __forceinline__ bool reaches(uint32_t w, uint32_t bound) { return __uint_as_float(w) >= __uint_as_float(bound); }
    static constexpr int kOf = 1;  // elements of a word
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int i) { return __uint_as_float(w[i]); }
};
template <typename T, typename T2> struct Halves {
    static constexpr int E = 8;
    static __device__ __forceinline__ T2 two(uint32_t w) {
        T2 r;
        memcpy(&r, &w, 4);
        return r;
    }
    static __device__ __forceinline__ uint32_t word(T2 v) {
        uint32_t r;
        memcpy(&r, &v, 4);
        return r;
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return word(__hmax2(two(a), two(b))); }
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int i) {
        return to_float(i & 1 ? two(w[i / 2]).y : two(w[i / 2]).x);
    }
    static __device__ __forceinline__ float one(uint32_t w) { return fmaxf(to_float(two(w).x), to_float(two(w).y)); }
    static __device__ __forceinline__ bool reaches(uint32_t w, uint32_t bound) { return !__hblt2(two(w), two(bound)); }
    static constexpr int kOf = 2;
};
template <> struct Pieces<__nv_bfloat16> : Halves<__nv_bfloat16, __nv_bfloat162> {
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int i) {
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    static constexpr uint32_t kNothing = 0xff80ff80u;
    static __device__ __forceinline__ uint32_t bound(float z) { return word(__bfloat162bfloat162(__float2bfloat16_rd(z))); }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) { return larger(w, kNothing); }
};
template <> struct Pieces<__half> : Halves<__half, __half2> {
    static constexpr uint32_t kNothing = 0xfc00fc00u;
    static __device__ __forceinline__ uint32_t bound(float z) { return word(__half2half2(__float2half_rd(z))); }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) { return larger(w, kNothing); }
};

template <typename T> __device__ __forceinline__ void beam_slice(const BeamArgs &a, int slice, int64_t k, int64_t b) {
    using P = Pieces<T>;
    constexpr int E = P::E;
    __shared__ float maxima[kBeamThreads];
    __shared__ uint64_t found[kFound];
    __shared__ float sums[kBeamWarps], tops[kBeamWarps];
    __shared__ uint64_t keys[kBeamThreads], bound_key;
    __shared__ int n_found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = b * a.K + k, slot = row * a.slices + slice;
    if (!alive(a, row)) return;  // its slots are not read
    const T *line = (const T *)a.logits + b * a.row + k * a.beam;
    // elements go to threads by their index, wherever the row begins: rows that are equal
    // have equal sums
    const int e0 = slice * kSlice<T>;
    const bool whole = ((uintptr_t)line & 15) == 0 && e0 + kSlice<T> <= a.V;
    // piece j of this thread, NaN as -inf, and -inf behind the row
    auto fetch = [&](int j, uint32_t (&w)[4]) {
        const int e = e0 + (j * kBeamThreads + tid) * E;
        if (!whole && e0 + j * kBeamThreads * E >= a.V) {  // for all of the CTA
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = P::kNothing;
        } else if (whole || e + E <= a.V) {
            const uint4 u = whole ? *(const uint4 *)(line + e) : load_vec<T>(line, e, a.V);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            alignas(16) T t[E];
#pragma unroll
            for (int i = 0; i < E; ++i) t[i] = e + i < a.V ? line[e + i] : from_float<T>(neg_inf());
            memcpy(w, t, 16);
        }
    };
    uint32_t w[kBeamVecs][4], larger[kBeamVecs], all_larger;
#pragma unroll
    for (int j = 0; j < kBeamVecs; ++j) fetch(j, w[j]);
#pragma unroll
    for (int j = 0; j < kBeamVecs; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[j][i] = P::clean(w[j][i]);
        larger[j] = P::larger(P::larger(w[j][0], w[j][1]), P::larger(w[j][2], w[j][3]));
        all_larger = j ? P::larger(all_larger, larger[j]) : larger[j];
    }
    const float most = P::one(all_larger);
    maxima[tid] = most;
    float top = most;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    if (tid == 0) n_found = 0;
    __syncthreads();
    // a larger key is a larger logit or, of equal ones, a lower token
    auto key = [&](float z, int token) { return (uint64_t)ordered(z) << 32 | (0xffffffffu - (uint32_t)token); };
    // Hands in all of this thread's that reach `least` (of keys), from the pieces whose largest
    // does; `bound` is its logit, or lower.
    auto gather = [&](uint64_t least, float bound) {
        const uint32_t low = P::bound(bound);
        uint32_t some = 0;
#pragma unroll
        for (int j = 0; j < kBeamVecs; ++j) some |= (uint32_t)P::reaches(larger[j], low) << j;
        while (some) {
            const int j = __ffs(some) - 1;
            some &= some - 1;
            uint32_t p[4];
            fetch(j, p);
            const int e = e0 + (j * kBeamThreads + tid) * E;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!P::reaches(P::clean(p[i]), low)) continue;
#pragma unroll
                for (int h = 0; h < P::kOf; ++h) {
                    const float z = P::get(p, i * P::kOf + h);
                    const uint64_t q = z > neg_inf() ? key(z, e + i * P::kOf + h) : 0;
                    if (q < least) continue;
                    const int at = atomicAdd(&n_found, 1);
                    if (at < kFound) found[at] = q;
                }
            }
        }
    };
    bool close = a.beams > 32;
    if (!close && warp == 0) {
        float group = maxima[lane];
#pragma unroll
        for (int i = 1; i < kBeamWarps; ++i) group = fmaxf(group, maxima[i * 32 + lane]);
        const uint32_t kth = kth_of_warp(group > neg_inf() ? ordered(group) : 0, a.beams);
        if (lane == 0) bound_key = kth ? (uint64_t)kth << 32 : 1;
    }
    // Exponentials relative to the warp's largest: at most 32 in a row are added in 32 bits,
    // then a thread's runs and the lanes; the warps and slices in 64.
    float sum = 0;
    if (fabsf(top) <= 1024.f) {
        // 2^(v log2(e) - c) with one operation before the power; what c lost to its rounding,
        // less than 10^-4 here, is a factor of the sum
        const float c = top * kLog2e, lost = fmaf(top, kLog2e, -c);
#pragma unroll
        for (int j = 0; j < kBeamVecs; j += 32 / E) {
            float run = 0;
#pragma unroll
            for (int q = j; q < j + 32 / E; ++q) {
                if (!whole && e0 + q * kBeamThreads * E >= a.V) continue;
#pragma unroll
                for (int i = 0; i < E; ++i) run += power(fmaf(P::get(w[q], i), kLog2e, -c));
            }
            sum += run;
        }
        sum *= power(-lost);
    } else if (fabsf(top) <= 3.402823466e38f) {
#pragma unroll 1
        for (int j = 0; j < kBeamVecs; ++j) {
            uint32_t p[4];
            fetch(j, p);
            float run = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = P::clean(p[i]);
#pragma unroll
            for (int i = 0; i < E; ++i) run += power((P::get(p, i) - top) * kLog2e);
            sum += run;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (!close) {
        const uint64_t least = bound_key;
        if (most > neg_inf()) gather(least, least > 1 ? unordered((uint32_t)(least >> 32)) : neg_inf());
        __syncthreads();
        close = n_found > kFew;
    }
    if (close) {
        uint64_t mine = 0;
#pragma unroll 1
        for (int j = 0; j < kBeamVecs; ++j) {
            uint32_t p[4];
            fetch(j, p);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float z = P::get(p, i);
                const uint64_t q = z > neg_inf() ? key(z, e0 + (j * kBeamThreads + tid) * E + i) : 0;
                mine = q > mine ? q : mine;
            }
        }
        keys[tid] = mine;
        __syncthreads();
        if (tid == 0) n_found = 0;
        if (warp == 0) {
            // the `beams`-th largest of the maxima, one after another
            uint64_t m[kBeamWarps];
#pragma unroll
            for (int i = 0; i < kBeamWarps; ++i) m[i] = keys[i * 32 + lane];
            uint64_t best = 0;
            for (int r = 0; r < a.beams; ++r) {
                uint64_t own = 0;
#pragma unroll
                for (int i = 0; i < kBeamWarps; ++i) own = own > m[i] ? own : m[i];
                const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(own >> 32));
                const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(own >> 32) == hi ? (uint32_t)own : 0u);
                best = (uint64_t)hi << 32 | lo;
                if (best == 0) break;  // no more than r threads have any: all of theirs are wanted
#pragma unroll
                for (int i = 0; i < kBeamWarps; ++i)
                    if (m[i] == best) m[i] = 0;
            }
            if (lane == 0) bound_key = best ? best : 1;
        }
        __syncthreads();
        if (mine >= bound_key) gather(bound_key, bound_key > 1 ? unordered((uint32_t)(bound_key >> 32)) : neg_inf());
        __syncthreads();
    }
    const int n = n_found;
    for (int i = tid; i < n; i += kBeamThreads) {
        const uint64_t q = found[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += found[j] > q;
        if (rank < a.beams) {
            a.value[slot * a.beams + rank] = unordered((uint32_t)(q >> 32));
            a.token[slot * a.beams + rank] = (int)(0xffffffffu - (uint32_t)q);
        }
    }
    if (warp == kBeamWarps - 1) {
        const bool some = lane < kBeamWarps;
        const float t = some ? tops[lane] : neg_inf();
        float all = t;
#pragma unroll
        for (int o = 4; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
        double s = some && t > neg_inf() && all <= 3.402823466e38f ? (double)sums[lane] * (double)expf(t - all) : 0;
#pragma unroll
        for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            a.sum[slot] = s;
            a.top[slot] = all;
            a.count[slot] = n < a.beams ? n : a.beams;
        }
    }
}

template <typename T> __global__ void __launch_bounds__(kBeamThreads, 4) k_beam_slices(const __grid_constant__ BeamArgs a) {
    beam_pdl_wait();
    beam_pdl_launch();
    beam_slice<T>(a, blockIdx.x, blockIdx.y, blockIdx.z);
}

// A candidate of a sequence: larger is better.
struct Head {
    uint64_t score;  // 0: none
    uint32_t beam, token;
    int list;
    __device__ __forceinline__ bool beats(const Head &o) const {
        if (score != o.score) return score > o.score;
        return beam != o.beam ? beam < o.beam : token < o.token;
    }
};

__device__ __forceinline__ Head best_of_warp(Head h) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        Head p;
        p.score = __shfl_xor_sync(0xffffffffu, h.score, o);
        p.beam = __shfl_xor_sync(0xffffffffu, h.beam, o);
        p.token = __shfl_xor_sync(0xffffffffu, h.token, o);
        p.list = __shfl_xor_sync(0xffffffffu, h.list, o);
        if (p.beats(h)) h = p;
    }
    return h;
}

__device__ __forceinline__ void beam_pick(const BeamArgs &a, int64_t b) {
    extern __shared__ uint8_t place[];  // of each list: how many have been taken (64 beams of 2,048 slices at most)
    __shared__ double base[kMostBeams];  // what a row's logits are added to
    __shared__ float about[kMostBeams];  // the same in 32 bits
    __shared__ uint8_t state[kMostBeams];  // 0 nothing, 1 by logits, 2 ended
    __shared__ Head heads[2][kBeamWarps];
    __shared__ uint64_t found_score[kFew], found_place[kFew];
    __shared__ float found_value[kFew];
    __shared__ uint32_t maxima[kBeamThreads * kAhead];
    __shared__ int n_found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = (int)a.K, lists = K * a.slices;
    if (tid == 0) n_found = 0;
    // Where there are not many lists, the first places of each are asked for before it is
    // known which rows' are looked at.  (The kernel is a chain of latencies, each of memory
    // some 0.4 us.)  Neighbouring threads take neighbouring lists, not places: the best are in
    // the first places, and groups that share them out bound best.
    const bool few_lists = lists <= kBeamThreads * kAhead && a.beams <= 32;
    int deep = few_lists ? kBeamThreads * kAhead / lists : 0;
    if (deep > a.beams) deep = a.beams;
    float value[kAhead];
    int token[kAhead], list[kAhead], at[kAhead], count[kAhead];
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
        at[r] = 0;
        list[r] = -1;
        const int i = tid + r * kBeamThreads;
        if (i >= lists * deep) continue;
        at[r] = i / lists;
        list[r] = i - at[r] * lists;
        const int64_t slot = b * lists + list[r];
        value[r] = load_l2(a.value + slot * a.beams + at[r]);
        token[r] = load_l2(a.token + slot * a.beams + at[r]);
        count[r] = load_l2(a.count + slot);
    }
    int width = 1;  // lanes of a row
    while (width < 32 && width < a.slices) width *= 2;
    const int sub = tid & (width - 1), at_once = kBeamThreads / width;
    for (int k0 = 0; k0 < K; k0 += at_once) {
        const int k = k0 + tid / width;
        const bool there = k < K;
        const int64_t row = b * K + (there ? k : 0), slot = row * a.slices;
        const float s = a.scores[row];
        const bool over = a.ended && a.ended[row];
        float first_top = neg_inf();
        double first_sum = 0;
        if (sub < a.slices) first_top = load_l2(a.top + slot + sub), first_sum = load_l2(a.sum + slot + sub);
        const bool finite = fabsf(s) <= 3.402823466e38f, looks = finite && !over;
        if (!looks) first_top = neg_inf();
        float top = first_top;
        double total = 0;
        if (looks)
            for (int i = sub + width; i < a.slices; i += width) top = fmaxf(top, load_l2(a.top + slot + i));
        for (int o = width / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool some = fabsf(top) <= 3.402823466e38f;
        if (some) {  // (a factor's error is one of 32 bits, as an exponential's)
            if (first_top > neg_inf()) total = first_sum * (double)expf(first_top - top);
            for (int i = sub + width; i < a.slices; i += width) total += load_l2(a.sum + slot + i) * (double)expf(load_l2(a.top + slot + i) - top);
        }
        for (int o = width / 2; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (sub == 0 && there) {
            state[k] = looks ? some : finite ? 2 : 0;
            const double d = !looks ? (double)s : some ? (double)s - ((double)top + log_of_sum(total)) : 0;
            base[k] = d;
            about[k] = (float)d;
        }
    }
    __syncthreads();
    // the candidate at place `at` of list l
    auto head_of = [&](int l, int at) {
        Head h{0, 0, 0, l};
        const int k = l / a.slices, s = l - k * a.slices;
        h.beam = (uint32_t)k;
        if (state[k] == 2) {
            if (s == 0 && at == 0) h.score = ordered(base[k]), h.token = (uint32_t)a.end_token;
        } else if (state[k] == 1) {
            const int64_t slot = b * lists + l;
            if (at < load_l2(a.count + slot)) {
                h.score = ordered(base[k] + (double)load_l2(a.value + slot * a.beams + at));
                h.token = (uint32_t)load_l2(a.token + slot * a.beams + at);
            }
        }
        return h;
    };
    auto put = [&](int r, const Head &h) {
        const int64_t at = b * a.beams + r;
        const bool some = h.score != 0;
        a.scores_out[at] = some ? (float)unordered(h.score) : neg_inf();
        a.parents[at] = some ? (int64_t)h.beam : r < K ? r : 0;
        a.tokens[at] = some ? (int64_t)h.token : -1;
        a.ended_out[at] = some && (int64_t)h.token == a.end_token;
    };
    if (few_lists) {
        // Sums in 32 bits, with what they may be off by, tell which candidates can be among the
        // best: there are few units for 64 bits.
        auto off_by = [&](int k, float sum) { return 1.2e-7f * (fabsf(about[k]) + fabsf(sum)); };
        auto can_reach = [&](int k, float v, float bound) {
            const float sum = about[k] + v;
            return !(sum + off_by(k, sum) < bound);
        };
        auto hand_in = [&](int k, float v, int token) {
            const int to = atomicAdd(&n_found, 1);
            if (to < kFew) found_value[to] = v, found_place[to] = (uint64_t)k << 32 | (uint32_t)token;
            return to < kFew;
        };
        int row_of[kAhead];
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            row_of[r] = -1;
            // A warp's candidates are shared out to the groups in an order that its places turn, so
            // that one row's first places in several groups are followed by its second in others.
            const int first = warp * 32 + r * kBeamThreads, turn = a.slices * (first / lists);
            uint32_t &mine = maxima[first + ((lane + turn) & 31)];
            mine = 0;
            if (list[r] < 0) continue;
            const int k = list[r] / a.slices, st = state[k];
            if (st == 2) value[r] = 0.f, token[r] = (int)a.end_token;
            if (st == 2 ? at[r] == 0 && list[r] == k * a.slices : st == 1 && at[r] < count[r]) {
                row_of[r] = k;
                const float sum = about[k] + value[r], off = off_by(k, sum);
                mine = ordered(off <= 3.402823466e38f ? sum - off : neg_inf());
            }
        }
        __syncthreads();
        uint32_t group = 0;
#pragma unroll
        for (int i = 0; i < kBeamWarps * kAhead; ++i) {
            const uint32_t m = maxima[i * 32 + lane];
            group = group > m ? group : m;
        }
        const uint32_t kth = kth_of_warp(group, a.beams);
        const float bound = kth ? unordered(kth) : neg_inf();
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            if (row_of[r] < 0 || !can_reach(row_of[r], value[r], bound)) continue;
            bool more = hand_in(row_of[r], value[r], token[r]) && at[r] == deep - 1 && state[row_of[r]] == 1;
            for (int next = deep; more && next < count[r]; ++next) {
                const int64_t slot = (b * lists + list[r]) * a.beams + next;
                const float v = load_l2(a.value + slot);
                more = can_reach(row_of[r], v, bound) && hand_in(row_of[r], v, load_l2(a.token + slot));
            }
        }
        __syncthreads();
        const int n = n_found;
        if (n <= kFew) {
            for (int i = tid; i < n; i += kBeamThreads) found_score[i] = ordered(base[found_place[i] >> 32] + (double)found_value[i]);
            __syncthreads();
            // four lanes rank a candidate
            for (int i0 = 0; i0 < n; i0 += kBeamThreads / 4) {
                const int i = i0 + tid / 4;
                const uint64_t score = i < n ? found_score[i] : 0, mine = i < n ? found_place[i] : 0;
                int rank = 0;
                for (int j = tid & 3; j < n; j += 4) rank += found_score[j] > score || (found_score[j] == score && found_place[j] < mine);
                rank += __shfl_xor_sync(0xffffffffu, rank, 1);
                rank += __shfl_xor_sync(0xffffffffu, rank, 2);
                if (i < n && rank < a.beams && (tid & 3) == 0) put(rank, Head{score, (uint32_t)(mine >> 32), (uint32_t)mine, 0});
            }
            for (int r = n + tid; r < a.beams; r += kBeamThreads) put(r, Head{0, 0, 0, 0});
            return;
        }
    }
    // one after another
    for (int i = tid; i < lists; i += kBeamThreads) place[i] = 0;
    auto best_of_mine = [&]() {
        Head best{0, 0, 0, -1};
        for (int l = tid; l < lists; l += kBeamThreads) {
            const Head h = head_of(l, place[l]);
            if (h.score && h.beats(best)) best = h;
        }
        return best;
    };
    Head mine = best_of_mine();
    for (int r = 0; r < a.beams; ++r) {
        const Head w = best_of_warp(mine);
        if (lane == 0) heads[r & 1][warp] = w;
        __syncthreads();
        Head best = heads[r & 1][0];
#pragma unroll
        for (int i = 1; i < kBeamWarps; ++i)
            if (heads[r & 1][i].beats(best)) best = heads[r & 1][i];
        if (tid == 0) put(r, best);
        if (best.score && best.list == mine.list) {
            ++place[best.list];
            mine = best_of_mine();
        }
    }
}

__global__ void __launch_bounds__(kBeamThreads, 4) k_beam_pick(const __grid_constant__ BeamArgs a) {
    beam_pdl_wait();
    beam_pdl_launch();
    beam_pick(a, blockIdx.x);
}

// Both in one, where a cluster holds a sequence's slices: its first CTA picks when all have
// left theirs.
constexpr int kCluster = 8;
template <typename T> __global__ void __launch_bounds__(kBeamThreads, 3) k_beam_cluster(const __grid_constant__ BeamArgs a) {
    beam_pdl_wait();
    beam_pdl_launch();
    beam_slice<T>(a, blockIdx.x, blockIdx.y, blockIdx.z);
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0) beam_pick(a, blockIdx.z);
}

// Launches a kernel whose CTAs may take their places while the one before ends: each waits
// for that before it reads anything (8 x 8 beams over 32,000 tokens and their states: 17.4 us
// instead of 21.9).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 cluster, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kBeamThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster.x;
    attr[1].val.clusterDim.y = cluster.y;
    attr[1].val.clusterDim.z = cluster.z;
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct BeamSpace {
    int slices;
    size_t sum, top, count, value, token, bytes;
};

BeamSpace beam_space(int64_t dtype, int64_t B, int64_t K, int64_t V, int64_t beams) {
    BeamSpace s{};
    s.slices = (int)((V + slice_of(dtype) - 1) / slice_of(dtype));
    const size_t n = (size_t)(B * K) * s.slices;
    s.sum = 0;
    s.top = s.sum + n * 8;
    s.count = s.top + n * 4;
    s.value = s.count + n * 4;
    s.token = s.value + n * beams * 4;
    s.bytes = s.token + n * beams * 4;
    return s;
}

ck_status check_beam_sizes(int64_t dtype, int64_t B, int64_t K, int64_t V, int64_t beams) {
    if (!known_dtype(dtype)) return fail(CK_ERR_INVALID_ARG, "beam search: unknown dtype %lld", (long long)dtype);
    if (B < 0 || K < 1 || V < 1 || beams < 1) return fail(CK_ERR_INVALID_ARG, "beam search: sizes must be positive");
    if (K > kMostBeams || beams > kMostBeams || V >= ((int64_t)1 << 24) || B > 65535)
        return fail(CK_ERR_UNSUPPORTED, "beam search: more than 64 beams, 65535 sequences or 2^24 tokens");
    return CK_OK;
}

// -- states ----------------------------------------------------------------------------------

constexpr int kStates = 32;         // arrays of a launch
constexpr int kRowChunk = 8192;     // bytes of a row that a CTA moves at a time

struct StateList {
    ck_beam_state s[kStates];
    int64_t start[kStates + 1];  // the array's first chunk
    int32_t chunks[kStates];     // chunks of a row
    int8_t unit[kStates];        // bytes that all its addresses are multiples of
    int count;
    const int64_t *parents;
    int K, beams;
};

// kMoves words of each thread are under way before the first is stored.
template <typename W> __device__ __forceinline__ void move_row(const char *from, char *to, int n) {
    constexpr int kMoves = sizeof(W) >= 4 ? kRowChunk / kBeamThreads / (int)sizeof(W) : 8;
    const int words = n / (int)sizeof(W);
    for (int i = threadIdx.x; i < words; i += kMoves * kBeamThreads) {
        W v[kMoves];
#pragma unroll
        for (int m = 0; m < kMoves; ++m) {
            v[m] = W{};
            if (from && i + m * kBeamThreads < words) v[m] = __ldcs((const W *)from + i + m * kBeamThreads);
        }
#pragma unroll
        for (int m = 0; m < kMoves; ++m)
            if (i + m * kBeamThreads < words) ((W *)to)[i + m * kBeamThreads] = v[m];
    }
}

// Rows from one array to another: a CTA takes a piece of one row.
__global__ void __launch_bounds__(kBeamThreads) k_reorder(const __grid_constant__ StateList a) {
    beam_pdl_wait();
    beam_pdl_launch();
    const int64_t c = blockIdx.x;
    int i = 0;
    while (c >= a.start[i + 1]) ++i;
    const ck_beam_state &s = a.s[i];
    const int64_t rows = (c - a.start[i]) / a.chunks[i], piece = (c - a.start[i]) - rows * a.chunks[i];
    const int64_t b = rows / a.beams, j = rows - b * a.beams;
    const int64_t p = a.parents[b * a.beams + j];
    const int64_t at = piece * kRowChunk;
    const int n = (int)(s.bytes - at < kRowChunk ? s.bytes - at : kRowChunk);
    const char *from = p >= 0 && p < a.K ? (const char *)s.in + b * s.in_row + p * s.in_beam + at : nullptr;
    char *to = (char *)s.out + b * s.out_row + j * s.out_beam + at;
    switch (a.unit[i]) {
        case 16: move_row<uint4>(from, to, n); break;
        case 8: move_row<uint2>(from, to, n); break;
        case 4: move_row<uint32_t>(from, to, n); break;
        case 2: move_row<uint16_t>(from, to, n); break;
        default: move_row<uint8_t>(from, to, n);
    }
}

// In place: a CTA takes the same piece of all rows of a sequence through shared memory.
template <typename W> __device__ __forceinline__ void move_rows(const StateList &a, const ck_beam_state &s, int64_t b,
                                                                int64_t at, int n, W *held) {
    const int words = n / (int)sizeof(W);
    for (int i = threadIdx.x; i < a.K * words; i += kBeamThreads) {
        const int k = i / words, w = i - k * words;
        held[i] = ((const W *)((const char *)s.in + b * s.in_row + k * s.in_beam + at))[w];
    }
    __syncthreads();
    const W zero{};
    for (int i = threadIdx.x; i < a.beams * words; i += kBeamThreads) {
        const int j = i / words, w = i - j * words;
        const int64_t p = a.parents[b * a.beams + j];
        if (p == j) continue;
        ((W *)((char *)s.out + b * s.out_row + j * s.out_beam + at))[w] = p >= 0 && p < a.K ? held[p * words + w] : zero;
    }
}

__global__ void __launch_bounds__(kBeamThreads, 4) k_reorder_in_place(const __grid_constant__ StateList a, int piece_bytes) {
    __shared__ uint4 held[32768 / 16];
    beam_pdl_wait();
    beam_pdl_launch();
    const int64_t c = blockIdx.x;
    int i = 0;
    while (c >= a.start[i + 1]) ++i;
    const ck_beam_state &s = a.s[i];
    const int64_t b = (c - a.start[i]) / a.chunks[i], piece = (c - a.start[i]) - b * a.chunks[i];
    const int64_t at = piece * piece_bytes;
    const int n = (int)(s.bytes - at < piece_bytes ? s.bytes - at : piece_bytes);
    switch (a.unit[i]) {
        case 16: move_rows(a, s, b, at, n, held); break;
        case 8: move_rows(a, s, b, at, n, (uint2 *)held); break;
        case 4: move_rows(a, s, b, at, n, (uint32_t *)held); break;
        case 2: move_rows(a, s, b, at, n, (uint16_t *)held); break;
        default: move_rows(a, s, b, at, n, (uint8_t *)held);
    }
}

int unit_of(const ck_beam_state &s) {
    const uintptr_t all = (uintptr_t)s.in | (uintptr_t)s.out | (uintptr_t)s.bytes | (uintptr_t)s.in_row |
                          (uintptr_t)s.in_beam | (uintptr_t)s.out_row | (uintptr_t)s.out_beam;
    for (int u = 16; u > 1; u /= 2)
        if (all % u == 0) return u;
    return 1;
}

// The bytes from an array's first to its last, [lo, hi); strides are not negative, and 0 along an
// axis of one.
struct Extent {
    uintptr_t lo, hi;
    bool written;
    int64_t row, beam, rows, beams, bytes;
    // The bytes that it takes of every m, from where it begins on, or more than m.
    int64_t of_every(int64_t m) const {
        int64_t n = bytes;
        for (const auto [stride, count] : {std::pair<int64_t, int64_t>{row, rows}, {beam, beams}})
            if (stride % m) n = stride < m ? n + (count - 1) * stride : m + 1;
        return n;
    }
    // Whether another, that begins no earlier, takes others of every so many bytes: columns of
    // one array, or halves of its sequences.
    bool beside(const Extent &o) const {
        for (const int64_t m : {row, beam, o.row, o.beam}) {
            if (m <= 0) continue;
            const int64_t apart = (int64_t)((o.lo - lo) % (uintptr_t)m);
            if (apart >= of_every(m) && o.of_every(m) <= m - apart) return true;
        }
        return false;
    }
};
Extent extent_of(const void *p, int64_t row, int64_t beam, int64_t B, int64_t n, int64_t bytes, bool written) {
    if (B == 1) row = 0;
    if (n == 1) beam = 0;
    return Extent{(uintptr_t)p, (uintptr_t)p + (uintptr_t)((B - 1) * row + (n - 1) * beam + bytes), written, row, beam, B, n, bytes};
}

// Whether what is written for one array is read or written for another.
bool states_tangled(std::vector<Extent> &all) {
    std::sort(all.begin(), all.end(), [](const Extent &x, const Extent &y) { return x.lo < y.lo; });
    for (size_t i = 0; i < all.size(); ++i)
        for (size_t j = i + 1; j < all.size() && all[j].lo < all[i].hi; ++j)
            if ((all[i].written || all[j].written) && !all[i].beside(all[j])) return true;
    return false;
}

ck_status check_states(const ck_beam_state *list, int64_t count, const int64_t *parents, int64_t B, int64_t K, int64_t beams) {
    if (count < 0 || (count && !list)) return fail(CK_ERR_INVALID_ARG, "states: no list");
    if (B < 0 || K < 1 || beams < 1) return fail(CK_ERR_INVALID_ARG, "states: sizes must be positive");
    if (K > kMostBeams || beams > kMostBeams || B > 65535)
        return fail(CK_ERR_UNSUPPORTED, "states: more than 64 beams or 65535 sequences");
    if (B == 0 || count == 0) return CK_OK;
    if (!parents) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(parents, 8)) return fail(CK_ERR_INVALID_ARG, "states: a pointer is not aligned to its elements");
    std::vector<Extent> all;
    all.reserve(2 * (size_t)count + 1);
    for (int64_t i = 0; i < count; ++i) {
        const ck_beam_state &s = list[i];
        if (s.bytes < 0 || s.in_row < 0 || s.in_beam < 0 || s.out_row < 0 || s.out_beam < 0)
            return fail(CK_ERR_INVALID_ARG, "states: negative size or stride");
        if (s.bytes == 0) continue;
        if (!s.in || !s.out) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
        // rows of out that share memory would be written in any order
        const int64_t n0 = B > 1 ? s.out_row : 0, n1 = beams > 1 ? s.out_beam : 0;
        const bool beams_inside = (beams == 1 || n1 >= s.bytes) && (B == 1 || n0 >= (beams - 1) * n1 + s.bytes);
        const bool rows_inside = (B == 1 || n0 >= s.bytes) && (beams == 1 || n1 >= (B - 1) * n0 + s.bytes);
        if (!beams_inside && !rows_inside) return fail(CK_ERR_INVALID_ARG, "states: rows of an output overlap");
        const bool own = s.in == s.out;
        if (own && (beams != K || (B > 1 && s.in_row != s.out_row) || (K > 1 && s.in_beam != s.out_beam)))
            return fail(CK_ERR_INVALID_ARG, "states: an array in its own place has the same strides and as many beams");
        all.push_back(extent_of(s.out, s.out_row, s.out_beam, B, beams, s.bytes, true));
        if (!own) all.push_back(extent_of(s.in, s.in_row, s.in_beam, B, K, s.bytes, false));
    }
    all.push_back(extent_of(parents, beams * 8, 8, B, beams, 8, false));
    if (states_tangled(all)) return fail(CK_ERR_INVALID_ARG, "states: an output overlaps another array or the parents");
    return CK_OK;
}

ck_status run_reorder(const ck_beam_state *list, int64_t count, const int64_t *parents, int64_t B, int64_t K,
                      int64_t beams, cudaStream_t s) {
    for (int in_place = 0; in_place < 2; ++in_place) {
        int piece = kRowChunk;
        while (in_place && piece * K > 32768) piece /= 2;
        StateList a{};
        a.parents = parents;
        a.K = (int)K;
        a.beams = (int)beams;
        auto flush = [&]() {
            if (!a.count) return cudaSuccess;
            const dim3 grid((unsigned)a.start[a.count]);
            a.count = 0;
            return in_place ? launch_early(k_reorder_in_place, grid, 1, 0, s, a, piece) : launch_early(k_reorder, grid, 1, 0, s, a);
        };
        cudaError_t e = cudaSuccess;
        for (int64_t i = 0; i < count && e == cudaSuccess; ++i) {
            if (!list[i].bytes || (list[i].in == list[i].out) != (in_place != 0)) continue;
            const int64_t per = (list[i].bytes + piece - 1) / piece, n = per * B * (in_place ? 1 : beams);
            if (per > 0x7fffffff || n > 0x7fffffff) return fail(CK_ERR_UNSUPPORTED, "states: rows too long");
            if (a.count == kStates || (a.count && a.start[a.count] + n > 0x7fffffff)) e = flush();
            if (e != cudaSuccess) break;
            a.s[a.count] = list[i];
            a.chunks[a.count] = (int32_t)per;
            a.unit[a.count] = (int8_t)unit_of(list[i]);
            a.start[a.count + 1] = (a.count ? a.start[a.count] : 0) + n;
            ++a.count;
        }
        if (e == cudaSuccess) e = flush();
        if (e != cudaSuccess) return cuda_fail(e, "k_reorder launch");
    }
    return CK_OK;
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_beam_workspace_size(int64_t dtype, int64_t B, int64_t K, int64_t V, int64_t beams, size_t *bytes) {
    const ck_status st = check_beam_sizes(dtype, B, K, V, beams);
    if (st != CK_OK) return st;
    if (!bytes) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    *bytes = beam_space(dtype, B, K, V, beams).bytes;
    return CK_OK;
}

extern "C" ck_status ck_beam_select(const ck_beam_call *c, void *stream) {
    if (!c) return fail(CK_ERR_INVALID_ARG, "beam search: no arguments");
    const ck_status st = check_beam_sizes(c->dtype, c->B, c->K, c->V, c->beams);
    if (st != CK_OK) return st;
    if (c->B == 0) return CK_OK;
    if (!c->logits || !c->scores || !c->scores_out || !c->parents || !c->tokens || !c->ended_out)
        return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (c->end_token < -1 || c->end_token >= c->V || (c->ended && c->end_token < 0))
        return fail(CK_ERR_INVALID_ARG, "beam search: end_token %lld is no token", (long long)c->end_token);
    if (!aligned(c->logits, dtype_size(c->dtype)) || !aligned(c->scores, 4) || !aligned(c->scores_out, 4) ||
        !aligned(c->parents, 8) || !aligned(c->tokens, 8) || !aligned(c->workspace, 8))
        return fail(CK_ERR_INVALID_ARG, "beam search: a pointer is not aligned to its elements");
    const BeamSpace sp = beam_space(c->dtype, c->B, c->K, c->V, c->beams);
    if (!c->workspace || (size_t)c->workspace_bytes < sp.bytes)
        return fail(CK_ERR_WORKSPACE, "beam search: a workspace of %zu bytes is needed", sp.bytes);
    BeamArgs a{};
    a.logits = c->logits;
    a.K = c->K, a.V = c->V, a.row = c->logits_row, a.beam = c->logits_beam;
    a.scores = c->scores, a.ended = c->ended, a.end_token = c->end_token;
    a.beams = (int)c->beams, a.slices = sp.slices;
    a.scores_out = c->scores_out, a.parents = c->parents, a.tokens = c->tokens, a.ended_out = c->ended_out;
    char *ws = (char *)c->workspace;
    a.sum = (double *)(ws + sp.sum), a.top = (float *)(ws + sp.top), a.count = (int *)(ws + sp.count);
    a.value = (float *)(ws + sp.value), a.token = (int *)(ws + sp.token);
    const cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid((unsigned)sp.slices, (unsigned)c->K, (unsigned)c->B);
    const size_t places = (size_t)c->K * sp.slices;  // a byte for each list
    if (places <= kCluster) {
        const cudaError_t e = with_dtype(c->dtype, [&](auto *tag) {
            return launch_early(k_beam_cluster<std::remove_pointer_t<decltype(tag)>>, grid, dim3(grid.x, grid.y), places, s, a);
        });
        return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_beam_cluster launch");
    }
    cudaError_t e = with_dtype(c->dtype, [&](auto *tag) {
        return launch_early(k_beam_slices<std::remove_pointer_t<decltype(tag)>>, grid, 1, 0, s, a);
    });
    if (e != cudaSuccess) return cuda_fail(e, "k_beam_slices launch");
    // (beside its other 13.5 KB the most that is had without asking is some 34 KB)
    constexpr int kMostPlaces = kMostBeams * (int)(((1 << 24) + kSlice<float> - 1) / kSlice<float>);
    static std::atomic<uint64_t> done;
    if (places > 32 * 1024) e = allow_smem((const void *)k_beam_pick, kMostPlaces, done);
    if (e == cudaSuccess) e = launch_early(k_beam_pick, dim3((unsigned)c->B), 1, places, s, a);
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_beam_pick launch");
}

extern "C" ck_status ck_reorder_states(const ck_beam_state *list, int64_t count, const int64_t *parents, int64_t B,
                                       int64_t K, int64_t beams, void *stream) {
    try {
        const ck_status st = check_states(list, count, parents, B, K, beams);
        if (st != CK_OK || B == 0 || count == 0) return st;
    } catch (const std::exception &) {
        return fail(CK_ERR_OUT_OF_MEMORY, "states: no host memory for %lld arrays", (long long)count);
    }
    return run_reorder(list, count, parents, B, K, beams, (cudaStream_t)stream);
}
