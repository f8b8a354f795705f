// ck_control_logits: penalties for repeated tokens, biases, grammar masks and
// temperature on a batch of logits, and in the same pass the next token.
#include <cstring>
#include <type_traits>

#include "ck_philox.h"
#include "ck_types.h"

namespace ck {
namespace {

// Threads of a CTA: four CTAs of the first kind fill an SM's registers, one of the second.
constexpr int kThreads1 = 256, kThreads4 = 1024, kLogitCtas = 4;
// Most tokens of a CTA, whose counts it holds in shared memory: in 16 bits each where the
// history is too short to count further, else in 32.
constexpr int kTile = 16256, kTileWide = 8064, kNarrow = 32767;
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

struct Row {
    float rep, freq, pres, temp;
    // A logit after the penalties, c what the table holds for its token.
    __device__ __forceinline__ float penalised(float z, uint32_t c) const {
        z = z > 0.f ? z / rep : z * rep;
        return __fsub_rn(z, __fadd_rn(__fmul_rn((float)(c >> 1), freq), c > 1 ? pres : 0.f));
    }
};

// For bounds; of numbers that are 0 or normal.
__device__ __forceinline__ float log2_fast(float v) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// z / t, rounded once, from q = z r with r = 1 / t and both t and r normal numbers.  A
// remainder times r, added to q, brings q within an ulp, a second one to the nearest
// float (P. W. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990), where remainders are exact; next to
// the ends of the type a division takes their place.  0, infinities and NaN are right in q.
// 64 x 131,072 fp32, sampled and returned, take 37 us so, 49 with a division for every
// token and 33 with q alone, which has a rounding too many.
__device__ __forceinline__ void quotients(float (&q)[kOct], const float (&z)[kOct], float t, float r) {
    constexpr float kLeast = 1e-30f, kMost = 8e37f;
    uint32_t ends = 0;
#pragma unroll
    for (int j = 0; j < kOct; ++j) {
        const float a = fabsf(z[j]), b = fabsf(q[j]);
        const bool plain = fminf(a, b) >= kLeast && b <= kMost;
        ends |= (uint32_t)(!plain && a > 0.f && a <= 3.402823466e38f) << j;
        float v = fmaf(fmaf(-q[j], t, z[j]), r, q[j]);
        v = fmaf(fmaf(-v, t, z[j]), r, v);
        q[j] = plain ? v : q[j];
    }
    if (ends) {
#pragma unroll
        for (int j = 0; j < kOct; ++j)
            if (ends >> j & 1) q[j] = z[j] / t;
    }
}

// Counts of the tokens that a CTA looks after: twice the number of occurrences in the
// history from `prompt` on, odd or not zero where the token was seen at all.  Additions
// of integers: their order does not matter.
struct Counts {
    uint32_t *slots;
    bool narrow;
    template <bool NARROW> __device__ __forceinline__ void put(uint32_t at, bool made) const {
        uint32_t *word = slots + (NARROW ? at >> 1 : at);
        const int up = NARROW ? (at & 1) * 16 : 0;
        if (made)
            atomicAdd(word, 2u << up);  // seen, and made here
        else
            atomicOr(word, 1u << up);
    }
    __device__ __forceinline__ uint32_t at(int o) const {
        return narrow ? ((const uint16_t *)slots)[o] : slots[o];
    }
    // a bit for each token of an oct that was seen
    __device__ __forceinline__ uint32_t seen(int o) const {
        uint32_t hit = 0;
        if (narrow) {
            const uint4 c = ((const uint4 *)slots)[o / 8];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                hit |= (uint32_t)((w[j] & 0xffff) != 0) << 2 * j | (uint32_t)(w[j] > 0xffff) << (2 * j + 1);
        } else {
            const uint4 c0 = ((const uint4 *)slots)[o / 4], c1 = ((const uint4 *)slots)[o / 4 + 1];
            const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) hit |= (uint32_t)(w[j] != 0) << j;
        }
        return hit;
    }
};

// Counts the tokens first <= v < first + span of history[0 .. len), len <= most, in slots
// from `slot` on.  The first ids are asked for before len is known; begin() empties the
// slots and says what len and prompt are.
template <int THREADS, bool NARROW, typename I, typename Begin>
__device__ __forceinline__ void count_history(const I *h, int most, uint32_t first, uint32_t span,
                                              const Counts &counts, int slot, Begin begin) {
    constexpr int kPer = 16 / (int)sizeof(I), kBatch = 4;  // ids of a load, loads on their way at once (8: 1 us more)
    int len = 0, prompt = 0;
    auto take = [&](I id, int i) {
        const uint32_t at = (uint32_t)id - first;
        if ((sizeof(I) == 4 || (uint64_t)id >> 32 == 0) && at < span && i < len)
            counts.put<NARROW>(slot + at, i >= prompt);
    };
    // single ids up to a 16-byte boundary and after the last
    int head = (int)((16 - ((uintptr_t)h & 15)) & 15) / (int)sizeof(I);
    if (head > most) head = most;
    const int pieces = (most - head) / kPer, tail = head + pieces * kPer;
    const uint4 *body = (const uint4 *)(h + head);
    for (int base = 0; base == 0 || (base < pieces && head + base * kPer < len); base += kBatch * THREADS) {
        const int i0 = base + threadIdx.x;
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (i0 + k * THREADS < pieces) v[k] = __ldg(body + i0 + k * THREADS);
        if (base == 0) {
            begin(len, prompt);
            if (threadIdx.x < head) take(__ldg(h + threadIdx.x), threadIdx.x);
            if (threadIdx.x < most - tail) take(__ldg(h + tail + threadIdx.x), tail + threadIdx.x);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * THREADS;
            if (i >= pieces || head + i * kPer >= len) break;
            I id[kPer];
            memcpy(id, &v[k], 16);
#pragma unroll
            for (int j = 0; j < kPer; ++j) take(id[j], head + i * kPer + j);
        }
    }
}

struct LogitPlan {
    int64_t slice;  // tokens of a CTA
    int slices;     // CTAs of a row
};

// A CTA takes a slice of a row's vocabulary, a thread eight tokens at a time, cut so
// that they are two blocks of the generator (sampling) or 16-byte pieces of the logits
// (else).  Where a row has several slices their best tokens go to `keys_out`, which
// k_pick looks through.
//
// What bounds it at large sizes is arithmetic: a token drawn costs a word of the
// generator, two logarithms and a division by the temperature.  All but the first are
// spared: as -log1p(-u) >= u, the noise is at most -log u, so a product and one
// approximate logarithm bound a score from above; a bound from below for a lane's
// likeliest token gives a score that the CTA's best has at least.  Only tokens that may
// reach it are scored as defined, and a lane puts its one off to the end, when few are
// left.  Bounds are a quarter of scores, which cannot overflow before the scores do
// (where those may, the bound is infinite, as infinite scores are equal),
// and leave out the scale of a word: log u = log word - 32 log 2.
//
// Measured: 64 x 131,072 bf16 with 4,096 of history, a bias, a mask and the logits wanted
// too, 36 MB in all: 32 us sampled (1.1 TB/s; 25 with 64 of history), 25 greedy at a
// temperature (41 with a division for each token), 22 with no token picked.  The
// instructions bound it: about 300 a warp and 256 tokens for the generator and the
// bounds, 150 for the rest, 140 for tokens of the history one by one.  That is with one
// wave of CTAs, whose counts have 16 bits; two waves of half the tokens take 36 us.
// 32 x 32,000 fp32 takes 9.9 us and 1 x 256 4.5, of which most is the launch and the way
// to memory, taken three times (ids, logits, the join's keys).
template <typename T, int PICK, int THREADS>
__global__ void __launch_bounds__(THREADS, kLogitCtas * kThreads1 / THREADS)
    k_logits(const __grid_constant__ ck_logit_call a, const __grid_constant__ PhiloxKeys keys, LogitPlan plan,
             unsigned long long *keys_out) {
    extern __shared__ __align__(16) uint32_t count[];
    __shared__ uint32_t floor_key;  // a score that some token of the CTA has at least
    __shared__ unsigned long long best_cta;
    const int64_t b = blockIdx.x / (unsigned)plan.slices;
    const int slice = (int)(blockIdx.x - (unsigned)b * plan.slices);
    const int64_t t0 = slice * plan.slice, t1 = t0 + plan.slice < a.V ? t0 + plan.slice : a.V;
    if (threadIdx.x == 0) best_cta = 0, floor_key = 0;
    const int64_t e0 = b * a.V;
    const T *row_in = (const T *)a.logits + b * a.logits_stride;
    // octs begin at tokens v with (v + cut) % 8 == 0; the oct at offset o holds tokens
    // v0 + o to v0 + o + 7, those with offsets in [from, to) there
    const int cut = PICK == kSample ? (int)(e0 & 7) : (int)(((uintptr_t)row_in / sizeof(T)) & 7);
    const int64_t v0 = t0 - cut;
    const int from = cut, to = cut + (int)(t1 - t0), octs = (to + kOct - 1) / kOct;
    const T *in = row_in + v0;
    T *out = a.out ? (T *)a.out + b * a.out_stride + v0 : nullptr;
    const float *bias = a.bias ? a.bias + b * a.bias_stride + v0 : nullptr;
    const uint32_t *mask = a.mask ? (const uint32_t *)a.mask + b * a.mask_stride : nullptr;
    const bool in_vec = ((uintptr_t)in & 15) == 0, out_vec = ((uintptr_t)out & 15) == 0,
               bias_vec = ((uintptr_t)bias & 15) == 0;
    // a thread's next oct, if it is all there: asked for while the one before is at work
    constexpr int kRaw = (int)sizeof(T) / 2;
    uint4 raw[kRaw];
    auto ask = [&](int ow) {
        const int o = (ow + (int)(threadIdx.x & 31)) * kOct;
        if (!in_vec || o < from || o + kOct > to) return;
#pragma unroll
        for (int i = 0; i < kRaw; ++i) raw[i] = __ldcs((const uint4 *)(in + o) + i);
    };
    const Counts counts{count, a.L <= kNarrow};
    const bool history = a.history && a.L > 0;
    if (history) {
        auto begin = [&](int &len, int &prompt) {
            len = (int)row_len(a.history_len, a.history_bits, b, a.L);
            prompt = a.prompt_len ? (int)row_len(a.prompt_len, a.history_bits, b, a.L) : 0;
            const int quads = counts.narrow ? octs : 2 * octs;
            for (int i = threadIdx.x; i < quads; i += THREADS) ((uint4 *)count)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        };
        auto count_all = [&](auto *tag) {
            const auto *h = (decltype(tag))a.history + b * a.history_stride;
            if (counts.narrow)
                count_history<THREADS, true>(h, (int)a.L, (uint32_t)t0, (uint32_t)(t1 - t0), counts, cut, begin);
            else
                count_history<THREADS, false>(h, (int)a.L, (uint32_t)t0, (uint32_t)(t1 - t0), counts, cut, begin);
        };
        if (a.history_bits == 32)
            count_all((const int32_t *)nullptr);
        else
            count_all((const int64_t *)nullptr);
    }
    ask(threadIdx.x & ~31);
    Row row;
    row.rep = a.repetition ? a.repetition[b] : a.repetition_all;
    row.freq = a.frequency ? a.frequency[b] : a.frequency_all;
    row.pres = a.presence ? a.presence[b] : a.presence_all;
    row.temp = a.temperature ? a.temperature[b] : a.temperature_all;
    const uint64_t step = PICK == kSample ? keys.at() : 0;
    __syncthreads();
    const bool heat = row.temp > 0.f;
    float cool = heat ? 1.f / row.temp : 1.f;
    // where the reciprocal is not precise the division comes first of all
    const float divide = !heat || (cool > 1e-37f && cool < 1e37f) ? 1.f : row.temp;
    if (divide != 1.f) row.temp = cool = 1.f;
    const float cool4 = cool * 0.25f;
    const bool bounded = heat && (PICK == kSample || row.temp != 1.f);
    unsigned long long best = 0;
    // a token that may be the one, to be scored when more is known; its logit before
    // the temperature
    float later_high = minus_inf(), later_z = 0.f;
    uint32_t later_word = 0;
    int later_o = 0;
    auto score_later = [&] {
        const float noise = PICK == kSample ? gumbel(later_word) : 0.f;
        const unsigned long long k = pick_key(__fadd_rn(later_z / row.temp, noise), (uint32_t)(v0 + later_o));
        best = k > best ? k : best;
    };
    // margins of bounds; NaN for what is -inf or NaN, and for +inf from below
    constexpr float kLog = 0.25f * 0.69314718f;  // a quarter of log 2
    // a quarter of the largest float, less more than a bound may be off: scores past it may
    // be infinite
    constexpr float kPast = 8.507e37f;
    auto above = [](float s) { return fmaf(fabsf(s), 1e-6f, s) + 1e-4f; };
    auto below = [](float s) { return fmaf(fabsf(s), -1e-6f, s) - 1e-4f; };
    for (int ow = threadIdx.x & ~31; ow < octs; ow += THREADS) {
        const int o = (ow + (int)(threadIdx.x & 31)) * kOct;
        const bool full = o >= from && o + kOct <= to;
        float z[kOct];
        uint32_t there = 0xff;  // tokens of the oct that exist
        if (full && in_vec) {
            alignas(16) T t[kOct];
#pragma unroll
            for (int i = 0; i < kRaw; ++i) ((uint4 *)t)[i] = raw[i];
#pragma unroll
            for (int j = 0; j < kOct; ++j) z[j] = to_float(t[j]);
        } else {
            there = 0;
#pragma unroll
            for (int j = 0; j < kOct; ++j) {
                const bool is = o + j >= from && o + j < to;
                z[j] = is ? to_float(in[o + j]) : minus_inf();  // never picked
                there |= (uint32_t)is << j;
            }
        }
        ask(ow + THREADS);
        // asked for here and used below
        float4 b0, b1;
        if (bias && full && bias_vec) b0 = *(const float4 *)(bias + o), b1 = *(const float4 *)(bias + o + 4);
        uint32_t allowed = ~0u;
        if (mask && full) {
            const int64_t v = v0 + o;
            const uint32_t *w = mask + (v >> 5);
            const int low = (int)(v & 31);
            allowed = __funnelshift_r(w[0], low > 32 - kOct ? w[1] : 0u, low);
        }
        if (history && there) {
            uint32_t hit = counts.seen(o);
            while (hit) {  // few: one by one
                const int at = __ffs(hit) - 1;
                hit &= hit - 1;
                float zv = 0.f;
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (j == at) zv = z[j];
                zv = row.penalised(zv, counts.at(o + at));
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (j == at) z[j] = zv;
            }
        }
        if (bias) {
            if (full && bias_vec) {
                const float bb[kOct] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
                for (int j = 0; j < kOct; ++j) z[j] = __fadd_rn(z[j], bb[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (there >> j & 1) z[j] = __fadd_rn(z[j], bias[o + j]);
            }
        }
        if (mask) {
            if (!full) {
                allowed = 0;
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (there >> j & 1) allowed |= (mask[(v0 + o + j) >> 5] >> ((v0 + o + j) & 31) & 1u) << j;
            }
#pragma unroll
            for (int j = 0; j < kOct; ++j)
                if (!(allowed >> j & 1)) z[j] = minus_inf();
        }
        if (divide != 1.f) {
#pragma unroll
            for (int j = 0; j < kOct; ++j) z[j] = z[j] / divide;
        }
        if (out) {
            // z / temperature; of 16 bits by a product, whose one more rounding of 32 bits these do not hold
            float q[kOct];
#pragma unroll
            for (int j = 0; j < kOct; ++j) q[j] = z[j] * cool;
            if (sizeof(T) == 4 && cool != 1.f) quotients(q, z, row.temp, cool);
            if (full && out_vec) {
                alignas(16) T t[kOct];
#pragma unroll
                for (int j = 0; j < kOct; ++j) t[j] = from_float<T>(q[j]);
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i) __stcs((uint4 *)(out + o) + i, ((const uint4 *)t)[i]);
            } else {
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (there >> j & 1) out[o + j] = from_float<T>(q[j]);
            }
        }
        if constexpr (PICK != kNone) {
            if (!bounded) {
                float top = minus_inf();
                int at = 0;
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (z[j] > top) top = z[j], at = j;  // of equal ones the first; no NaN
                const unsigned long long k = pick_key(top, (uint32_t)(v0 + o + at));
                best = k > best ? k : best;
                continue;
            }
            uint32_t w[kOct] = {};
            if constexpr (PICK == kSample) {
                uint4 r0, r1;
                philox_two((uint64_t)(e0 + v0 + o) >> 2, step, keys, r0, r1);
                w[0] = r0.x, w[1] = r0.y, w[2] = r0.z, w[3] = r0.w;
                w[4] = r1.x, w[5] = r1.y, w[6] = r1.z, w[7] = r1.w;
            }
            // a score is at most above(s) (errors of products and logarithms, the word as
            // a float and z / temperature as a product are in the margin)
            float s[kOct], top = minus_inf();
#pragma unroll
            for (int j = 0; j < kOct; ++j) {
                s[j] = PICK == kSample ? fmaf(log2_fast((float)w[j]), -kLog, z[j] * cool4) : z[j] * cool4;
                top = fmaxf(top, s[j]);
            }
            if (top > kPast) {  // infinite scores are equal: all that may be are scored
#pragma unroll
                for (int j = 0; j < kOct; ++j)
                    if (s[j] > kPast) s[j] = -minus_inf();
                top = -minus_inf();
            }
            const uint32_t seen = *(volatile uint32_t *)&floor_key;
            float floor = key_score((unsigned long long)seen << 32);
            if (!__any_sync(~0u, above(top) >= floor)) continue;
            // A score that a lane's likeliest token has at least: with t >= u,
            // -log1p(-u) <= t / (1 - t).
            int at = -1;
            float low = minus_inf(), z_at = 0.f;
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < kOct; ++j)
                if (s[j] == top) at = j, z_at = z[j], word = w[j];
            if constexpr (PICK == kSample) {
                const float t = fmaf((float)word, 1.0000003f, 1.f), rest = fmaf(t, -2.3283064365386963e-10f, 1.f);
                if (rest > 0.5f) low = below(fmaf(log2_fast(rest) - log2_fast(t), kLog, z_at * cool4));
            } else {
                low = below(top);
            }
            // (an unsigned word in the order of floats, as pick_key's upper one)
            const uint32_t warp_key = __reduce_max_sync(~0u, at < 0 ? 0 : (uint32_t)(pick_key(low, 0) >> 32));
            if (warp_key > seen) {
                if ((threadIdx.x & 31) == 0) atomicMax(&floor_key, warp_key);
                floor = key_score((unsigned long long)warp_key << 32);
            }
            while (above(top) >= floor) {
                // a token put off earlier, should it still be one to score, makes room
                if (later_high >= floor && later_high > minus_inf()) score_later();
                later_high = above(top);
                later_o = o + at;
                later_z = z_at;
                later_word = word;
                top = minus_inf();
                const int old = at;
#pragma unroll
                for (int j = 0; j < kOct; ++j) {
                    if (j == old) s[j] = minus_inf();
                    if (s[j] > top) top = s[j], at = j, z_at = z[j], word = w[j];
                }
            }
        }
    }
    if constexpr (PICK != kNone) {
        __syncthreads();  // the floor is known
        if (later_high > minus_inf() &&
            later_high >= key_score((unsigned long long)floor_key << 32))
            score_later();
        for (int o = 16; o; o >>= 1) {
            const unsigned long long k = __shfl_xor_sync(~0u, best, o);
            best = k > best ? k : best;
        }
        if ((threadIdx.x & 31) == 0 && best) atomicMax(&best_cta, best);
        __syncthreads();
        if (threadIdx.x == 0) {
            if (plan.slices > 1)
                keys_out[blockIdx.x] = best_cta;
            else
                a.tokens[b] = best_cta ? (int64_t)(0xFFFFFFFFu - (uint32_t)best_cta) : -1;
        }
    }
}

// The best of a row's slices, a warp for a row.
__global__ void __launch_bounds__(128) k_pick(const unsigned long long *keys, int slices, int64_t B, int64_t *tokens) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t b = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (b >= B) return;
    unsigned long long best = 0;
    for (int i = threadIdx.x & 31; i < slices; i += 32) best = keys[b * slices + i] > best ? keys[b * slices + i] : best;
    for (int o = 16; o; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(~0u, best, o);
        best = k > best ? k : best;
    }
    if ((threadIdx.x & 31) == 0) tokens[b] = best ? (int64_t)(0xFFFFFFFFu - (uint32_t)best) : -1;
}

// Slices of a row: as many CTAs as the device holds at once, or a whole number of
// times that, of as many tokens at most as the table has room for.  A CTA reads all of
// its row's history, so a slice is no smaller than a quarter of that; nor than 1,024
// tokens.  Up to kTileWide tokens a row stays whole where one is picked: a second kernel
// costs more.
LogitPlan logit_plan(int64_t B, int64_t V, int64_t L, bool pick, int sms) {
    const int64_t slots = (int64_t)sms * kLogitCtas, tile = L <= kNarrow ? kTile : kTileWide;
    const int64_t waves = (B * V + tile * slots - 1) / (tile * slots);
    int64_t slices = waves * slots / (B > 0 ? B : 1);
    int64_t least = L / 4 > 1024 ? L / 4 : 1024;
    if (least > tile) least = tile;
    if (slices > (V + least - 1) / least) slices = (V + least - 1) / least;
    if (slices < (V + tile - 1) / tile) slices = (V + tile - 1) / tile;
    if (pick && V <= kTileWide) slices = 1;
    const int64_t slice = ((V + slices - 1) / slices + 127) / 128 * 128;
    return LogitPlan{slice, (int)((V + slice - 1) / slice)};
}

template <typename T, int PICK>
cudaError_t launch_logits(const ck_logit_call &a, const PhiloxKeys &keys, const LogitPlan &plan,
                          cudaStream_t stream) {
    const size_t smem = a.history ? (size_t)(plan.slice + 2 * kOct) * (a.L <= kNarrow ? 2 : 4) : 0;
    // Where CTAs are no more than SMs and have much to read, one takes a whole SM: 20
    // rows of 50,021 tokens with 32,768 of history take 11 us so, 21 by 256 threads each.
    const unsigned ctas = (unsigned)(a.B * plan.slices);
    unsigned long long *best = (unsigned long long *)a.workspace;
    if (ctas <= (unsigned)device_sms() && (plan.slice >= 4096 || (a.history && a.L >= 4096)))
        k_logits<T, PICK, kThreads4><<<ctas, kThreads4, smem, stream>>>(a, keys, plan, best);
    else
        k_logits<T, PICK, kThreads1><<<ctas, kThreads1, smem, stream>>>(a, keys, plan, best);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || PICK == kNone || plan.slices == 1) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.B + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_pick, (const unsigned long long *)a.workspace, plan.slices, a.B, a.tokens);
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
    if (a.out && a.B > 1 && a.out_stride < a.V)
        return fail(CK_ERR_INVALID_ARG, "control_logits: the rows of out overlap");
    const size_t el = dtype_size(a.dtype), id = a.history && a.history_bits == 32 ? 4 : 8;
    if (!aligned(a.logits, el) || !aligned(a.out, el) || !aligned(a.tokens, 8) || !aligned(a.step_dev, 8) ||
        (a.history && (!aligned(a.history, id) || !aligned(a.history_len, id) || !aligned(a.prompt_len, id))) ||
        !aligned(a.repetition, 4) || !aligned(a.frequency, 4) || !aligned(a.presence, 4) ||
        !aligned(a.temperature, 4) || !aligned(a.bias, 4) || !aligned(a.mask, 4))
        return fail(CK_ERR_INVALID_ARG, "control_logits: a pointer is not aligned to its elements");
    const LogitPlan plan = logit_plan(a.B, a.V, a.history ? a.L : 0, a.tokens != nullptr, device_sms());
    if (a.B * (int64_t)plan.slices >= ((int64_t)1 << 31))
        return fail(CK_ERR_UNSUPPORTED, "control_logits: B V is too large");
    if (a.tokens && plan.slices > 1 &&
        (!a.workspace || ((uintptr_t)a.workspace & 7) != 0 || a.workspace_bytes < a.B * plan.slices * 8))
        return fail(CK_ERR_WORKSPACE, "control_logits: workspace of %lld bytes (%lld needed, 8-byte aligned)",
                    (long long)(a.workspace ? a.workspace_bytes : 0), (long long)(a.B * plan.slices * 8));
    const PhiloxKeys keys = PhiloxKeys::of(a.seed, a.step, a.step_dev);
    cudaError_t e = cudaSuccess;
    with_dtype(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        cudaStream_t s = (cudaStream_t)stream;
        e = !a.tokens  ? launch_logits<T, kNone>(a, keys, plan, s)
            : a.sample ? launch_logits<T, kSample>(a, keys, plan, s)
                       : launch_logits<T, kGreedy>(a, keys, plan, s);
    });
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_logits launch");
}

extern "C" ck_status ck_logits_workspace_size(int64_t B, int64_t V, int64_t L, size_t *bytes) {
    if (B < 0 || V < 1 || L < 0 || !bytes)
        return fail(CK_ERR_INVALID_ARG, "logits_workspace_size: B, L >= 0, V >= 1, bytes not NULL");
    const LogitPlan plan = logit_plan(B, V, L, true, device_sms());
    *bytes = plan.slices > 1 ? (size_t)B * plan.slices * 8 : 0;
    return CK_OK;
}
