// ck_beam_select: of a beam search's K V candidates for each sequence the best, and
// ck_reorder_states: the beams' states moved to the places of those that were kept.
//
// The selection reads the logits once.  A CTA takes a slice of a beam's row into registers
// and leaves the slice's maximum, its sum of exponentials and its best candidates: the
// score's other terms are the same for all of a row, so inside one the order is that of
// the logits.  A second kernel, a CTA for each sequence, joins the slices' sums and picks
// from the heads of their lists, with scores in 64 bits.
//
// A slice's best: the `beams`-th largest of the threads' maxima bounds them from below, as
// so many elements are at least that.  Only threads whose maximum reaches the bound look
// at their elements, and what they find is ranked by counting.
//
// What bounds it is memory for large vocabularies, latency for small ones.
#include <algorithm>
#include <vector>

#include "ck_types.h"

namespace ck {
namespace {

constexpr int kBeamThreads = 256, kBeamWarps = kBeamThreads / 32;
constexpr int kPer = 32;                          // elements of a thread
constexpr int kSlice = kBeamThreads * kPer;       // elements of a slice
constexpr int kMostBeams = 64;
constexpr int kMostLists = 40960;                 // beams times slices

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
    const float s = __ldg(a.scores + at);
    return fabsf(s) <= 3.402823466e38f && !(a.ended && __ldg(a.ended + at));
}

template <typename T> __global__ void __launch_bounds__(kBeamThreads) k_beam_slices(const __grid_constant__ BeamArgs a) {
    constexpr int E = 16 / (int)sizeof(T), kVecs = kPer / E;
    __shared__ uint64_t maxima[kBeamThreads];
    __shared__ uint64_t found[kMostBeams * kPer];
    __shared__ double sums[kBeamWarps];
    __shared__ float tops[kBeamWarps];
    __shared__ uint64_t bound;
    __shared__ int n_found;
    beam_pdl_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.z, k = blockIdx.y, row = b * a.K + k, slot = row * a.slices + blockIdx.x;
    if (!alive(a, row)) return;  // its slots are not read
    const T *line = (const T *)a.logits + b * a.row + k * a.beam;
    // elements go to threads by their index, wherever the row begins: rows that are equal
    // have equal sums
    const int e0 = blockIdx.x * kSlice;
    float v[kPer];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int e = e0 + (j * kBeamThreads + tid) * E;
        if (e + E <= a.V) {
            const uint4 w = load_vec<T>(line, e, a.V);
            alignas(16) T t[E];
            memcpy(t, &w, 16);
#pragma unroll
            for (int i = 0; i < E; ++i) v[j * E + i] = to_float(t[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[j * E + i] = e + i < a.V ? to_float(line[e + i]) : neg_inf();
        }
    }
    auto token_of = [&](int i) { return e0 + ((i / E) * kBeamThreads + tid) * E + i % E; };
    float most = neg_inf();
    int where = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (v[i] != v[i]) v[i] = neg_inf();
        if (v[i] > most) most = v[i], where = i;
    }
    // a larger key is a larger logit or, of equal ones, a lower token
    auto key = [&](float z, int token) { return (uint64_t)ordered(z) << 32 | (0xffffffffu - (uint32_t)token); };
    const uint64_t mine = most > neg_inf() ? key(most, token_of(where)) : 0;
    maxima[tid] = mine;
    float top = most;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    if (tid == 0) n_found = 0;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int w = 1; w < kBeamWarps; ++w) top = fmaxf(top, tops[w]);
    if (warp == 0) {
        // the `beams`-th largest of the maxima, one after another
        uint64_t m[kBeamWarps];
#pragma unroll
        for (int i = 0; i < kBeamWarps; ++i) m[i] = maxima[i * 32 + lane];
        uint64_t best = 0;
        for (int r = 0; r < a.beams; ++r) {
            uint64_t own = 0;
#pragma unroll
            for (int i = 0; i < kBeamWarps; ++i) own = own > m[i] ? own : m[i];
            const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(own >> 32));
            const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(own >> 32) == hi ? (uint32_t)own : 0u);
            best = (uint64_t)hi << 32 | lo;
            if (best == 0) break;  // no more than r elements: all of them are wanted
#pragma unroll
            for (int i = 0; i < kBeamWarps; ++i)
                if (m[i] == best) m[i] = 0;
        }
        if (lane == 0) bound = best ? best : 1;
    }
    double sum = 0;
    if (top > neg_inf()) {
        float s = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += __expf(v[i] - top);
        sum = s;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (mine >= bound) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint64_t q = key(v[i], token_of(i));
            if (v[i] > neg_inf() && q >= bound) found[atomicAdd(&n_found, 1)] = q;
        }
    }
    __syncthreads();
    const int n = n_found;
    for (int i = tid; i < n; i += kBeamThreads) {
        const uint64_t q = found[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += found[j] > q;
        if (rank < a.beams) {
            a.value[slot * a.beams + rank] = unordered((uint32_t)(q >> 32));
            a.token[slot * a.beams + rank] = (int)(0xffffffffu - (uint32_t)q);
        }
    }
    if (tid == 0) {
        double s = 0;
        for (int w = 0; w < kBeamWarps; ++w) s += sums[w];
        a.sum[slot] = s;
        a.top[slot] = top;
        a.count[slot] = n < a.beams ? n : a.beams;
    }
}

// A candidate at the head of a list: larger is better.
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

__global__ void __launch_bounds__(kBeamThreads) k_beam_pick(const __grid_constant__ BeamArgs a) {
    extern __shared__ uint8_t place[];  // of each list: how many have been taken
    __shared__ double base[kMostBeams];  // what a row's logits are added to
    __shared__ uint8_t state[kMostBeams];  // 0 nothing, 1 by logits, 2 ended
    __shared__ Head heads[2][kBeamWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x;
    const int lists = (int)a.K * a.slices;
    for (int i = tid; i < lists; i += kBeamThreads) place[i] = 0;
    beam_pdl_wait();
    for (int k = warp; k < a.K; k += kBeamWarps) {
        const int64_t row = b * a.K + k, slot = row * a.slices;
        const float s = __ldg(a.scores + row);
        const bool finite = fabsf(s) <= 3.402823466e38f;
        const bool over = a.ended && __ldg(a.ended + row);
        double total = 0;
        float top = neg_inf();
        if (finite && !over) {
            for (int i = lane; i < a.slices; i += 32) top = fmaxf(top, __ldcg(a.top + slot + i));
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const bool some = fabsf(top) <= 3.402823466e38f;
            if (some)
                for (int i = lane; i < a.slices; i += 32)
                    total += __ldcg(a.sum + slot + i) * exp((double)__ldcg(a.top + slot + i) - (double)top);
#pragma unroll
            for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (lane == 0) {
                state[k] = some;
                base[k] = some ? (double)s - ((double)top + log(total)) : 0;
            }
        } else if (lane == 0) {
            state[k] = finite ? 2 : 0;
            base[k] = s;
        }
    }
    __syncthreads();
    auto head_of = [&](int l) {
        Head h{0, 0, 0, l};
        const int k = l / a.slices, s = l - k * a.slices;
        const int at = place[l];
        h.beam = (uint32_t)k;
        if (state[k] == 2) {
            if (s == 0 && at == 0) h.score = ordered(base[k]), h.token = (uint32_t)a.end_token;
        } else if (state[k] == 1) {
            const int64_t slot = (b * a.K + k) * a.slices + s;
            if (at < __ldcg(a.count + slot)) {
                h.score = ordered(base[k] + (double)__ldcg(a.value + slot * a.beams + at));
                h.token = (uint32_t)__ldcg(a.token + slot * a.beams + at);
            }
        }
        return h;
    };
    auto best_of_mine = [&]() {
        Head best{0, 0, 0, -1};
        for (int l = tid; l < lists; l += kBeamThreads) {
            const Head h = head_of(l);
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
        if (tid == 0) {
            const int64_t at = b * a.beams + r;
            const bool some = best.score != 0;
            a.scores_out[at] = some ? (float)unordered(best.score) : neg_inf();
            a.parents[at] = some ? (int64_t)best.beam : r < a.K ? r : 0;
            a.tokens[at] = some ? (int64_t)best.token : -1;
            a.ended_out[at] = some && (int64_t)best.token == a.end_token;
        }
        if (best.score && best.list == mine.list) {
            ++place[best.list];
            mine = best_of_mine();
        }
    }
}

struct BeamSpace {
    int slices;
    size_t sum, top, count, value, token, bytes;
};

BeamSpace beam_space(int64_t B, int64_t K, int64_t V, int64_t beams) {
    BeamSpace s{};
    s.slices = (int)((V + kSlice - 1) / kSlice);
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
    // a byte of shared memory for each list
    if (K * beam_space(B, K, V, beams).slices > kMostLists)
        return fail(CK_ERR_UNSUPPORTED, "beam search: too many beams and tokens at once");
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

template <typename W> __device__ __forceinline__ void move_row(const char *from, char *to, int64_t n) {
    const W zero{};
    for (int64_t i = threadIdx.x; i * (int64_t)sizeof(W) < n; i += kBeamThreads)
        ((W *)to)[i] = from ? ((const W *)from)[i] : zero;
}

// Rows from one array to another: a CTA takes a piece of one row.
__global__ void __launch_bounds__(kBeamThreads) k_reorder(const __grid_constant__ StateList a) {
    const int64_t c = blockIdx.x;
    int i = 0;
    while (c >= a.start[i + 1]) ++i;
    const ck_beam_state &s = a.s[i];
    const int64_t rows = (c - a.start[i]) / a.chunks[i], piece = (c - a.start[i]) - rows * a.chunks[i];
    const int64_t b = rows / a.beams, j = rows - b * a.beams;
    const int64_t p = __ldg(a.parents + b * a.beams + j);
    const int64_t at = piece * kRowChunk, n = s.bytes - at < kRowChunk ? s.bytes - at : kRowChunk;
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
        const int64_t p = __ldg(a.parents + b * a.beams + j);
        if (p == j) continue;
        ((W *)((char *)s.out + b * s.out_row + j * s.out_beam + at))[w] = p >= 0 && p < a.K ? held[p * words + w] : zero;
    }
}

__global__ void __launch_bounds__(kBeamThreads) k_reorder_in_place(const __grid_constant__ StateList a, int piece_bytes) {
    __shared__ uint4 held[32768 / 16];
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

// The bytes from an array's first to its last, [lo, hi); strides are not negative.
struct Extent {
    uintptr_t lo, hi;
    bool written;
    int64_t row, beam, bytes;
    // Whether the two are columns of one array that do not meet.
    bool beside(const Extent &o) const {
        if (row != o.row || beam != o.beam || beam <= 0 || row % beam) return false;
        const int64_t d = (int64_t)((o.lo > lo ? o.lo - lo : lo - o.lo) % (uintptr_t)beam);
        const int64_t first = o.lo > lo ? bytes : o.bytes, second = o.lo > lo ? o.bytes : bytes;
        return d >= first && d + second <= beam;
    }
};
Extent extent_of(const void *p, int64_t row, int64_t beam, int64_t B, int64_t n, int64_t bytes, bool written) {
    return Extent{(uintptr_t)p, (uintptr_t)p + (uintptr_t)((B - 1) * row + (n - 1) * beam + bytes), written, row, beam, bytes};
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
    all.reserve(2 * (size_t)count);
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
    if (states_tangled(all)) return fail(CK_ERR_INVALID_ARG, "states: an output overlaps another array");
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
            if (in_place)
                k_reorder_in_place<<<(unsigned)a.start[a.count], kBeamThreads, 0, s>>>(a, piece);
            else
                k_reorder<<<(unsigned)a.start[a.count], kBeamThreads, 0, s>>>(a);
            a.count = 0;
            return cudaGetLastError();
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
    *bytes = beam_space(B, K, V, beams).bytes;
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
    const BeamSpace sp = beam_space(c->B, c->K, c->V, c->beams);
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
    with_dtype(c->dtype, [&](auto *tag) {
        k_beam_slices<std::remove_pointer_t<decltype(tag)>><<<grid, kBeamThreads, 0, s>>>(a);
    });
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "k_beam_slices launch");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)c->B);
    cfg.blockDim = dim3(kBeamThreads);
    cfg.dynamicSmemBytes = (size_t)c->K * sp.slices;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_beam_pick, a);
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
