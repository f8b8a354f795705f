// ck_dropout: dropout whose mask comes from a counter-based generator and is
// never stored.  The backward is the same call on the gradient: the element's
// index gives its word again.
#include <cmath>
#include <cstring>

#include "ck_philox.h"
#include "ck_types.h"

namespace ck {
namespace {

struct DropArgs {
    const void *x;
    void *y;
    int64_t rep, n1, n2, n3;              // the mask's elements [n1][n2][n3], used `rep` times
    int64_t xr, x1, x2, x3;               // element strides of x: repeat, then the mask's axes
    int64_t yr, y1, y2, y3;
    uint32_t threshold;                   // keep an element whose word is >= threshold
    int drop_all;                         // p = 1: read as zeros (scale is 0 too)
    float scale;
    PhiloxKeys keys;
};

// Any strides, element by element: for an innermost axis of x that is not dense.
// 64 x 32 x 5,000 fp32 take 74 us with the last two axes swapped, 69 as every second
// element and 60 as one number repeated; the divisions of an element's index and, of
// the first, sectors read for four bytes of them bound it.
//
// A select and not a product: a dropped element is 0 whatever it held.
template <typename T>
__global__ void __launch_bounds__(256) k_dropout(const __grid_constant__ DropArgs a) {
    const uint64_t step = a.keys.at();
    const T *x = (const T *)a.x;
    T *y = (T *)a.y;
    const int64_t n = a.n1 * a.n2 * a.n3, blocks = (n + 3) / 4;
    for (int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; q < blocks;
         q += (int64_t)gridDim.x * blockDim.x) {
        const uint4 r = philox((uint64_t)q, step, a.keys);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = 4 * q + j;
            if (m >= n) break;
            const int64_t i3 = m % a.n3, t = m / a.n3, i2 = t % a.n2, i1 = t / a.n2;
            const bool keep = !a.drop_all && w[j] >= a.threshold;
            for (int64_t k = 0; k < a.rep; ++k) {
                const float v = to_float(x[k * a.xr + i1 * a.x1 + i2 * a.x2 + i3 * a.x3]);
                y[k * a.yr + i1 * a.y1 + i2 * a.y2 + i3 * a.y3] =
                    from_float<T>(keep ? v * a.scale : 0.f);
            }
        }
    }
}


// Where x's innermost axis is dense and y is dense and aligned, a thread takes 16
// bytes of y: E elements whose words are those of E / 4 of the generator's blocks,
// as y is dense in the order of the mask.  What bounds it is memory, every element read
// and written once, with the generator close behind: a block is twenty 32 x 32 -> 64
// bit products for four elements, of which an SM does 0.1 a nanosecond for each of 32 lanes.
//
// Measured: k_dropout_dense on 32 x 256 x 20,000 bf16 131 us (5.0 TB/s; the blocks alone
// 86), k_dropout_lines on 64 x 32 x 5,000 fp32 with one mask 14 us (5.8 TB/s),
// k_dropout_flat on 32 x 20 x 4,999 fp16 cut out of wider rows 6.5 us (1.95 TB/s: a
// start, one way to memory and back, and an end), 8 x 8 x 256 fp32 1.5 us.
constexpr int kDropThreads = 256;

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", PLDI 1994).
struct Divider {
    uint32_t d, mul, shift;
    static Divider of(uint32_t d) {
        uint32_t s = 0;
        while (((uint64_t)1 << s) < d) ++s;
        return Divider{d, (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1), s};
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
};

struct DropFlat {
    DropArgs a;
    int64_t n;             // elements of y
    int64_t period;        // locked: elements of the mask, else n
    Divider row, plane;    // n3 and n2 (for n < 2^31)
    int small;             // n < 2^31
    int rows_joined;       // rows n3 apart: x is one dense line
};

// Elements e .. e + E - 1 of a dense line at p + e (element e itself there), of which
// `room` are there, whatever p's alignment: from the two aligned 16-byte pieces that
// hold them, where both lie inside the line, else one by one.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T *line, int64_t e, int64_t length) {
    constexpr int E = kVec<T>;
    const T *p = line + e;
    const uint32_t off = (uint32_t)(uintptr_t)p & 15u;
    if (off == 0) return __ldcs((const uint4 *)p);
    const uint4 *lo = (const uint4 *)((uintptr_t)p - off);
    if ((const char *)lo >= (const char *)line && (const char *)(lo + 2) <= (const char *)(line + length)) {
        const uint4 u = __ldg(lo), v = __ldg(lo + 1);
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

// Where in the generator's blocks of four a piece of E elements begins.
enum Start {
    kPiece,  // at a multiple of E
    kBlock,  // at a multiple of four
    kWithin  // anywhere
};

// Which of a piece's E elements are kept.
template <typename T> struct Keep {
    bool k[kVec<T>];
    // elements m .. m + E - 1 of the mask
    template <int START>
    __device__ __forceinline__ void make(const DropArgs &a, uint64_t step, int64_t m) {
        constexpr bool SHIFTED = START == kWithin;
        constexpr int E = kVec<T>, kBlocks = E / 4 + (SHIFTED ? 1 : 0);
        uint4 r[kBlocks];
        if constexpr (START == kPiece && kBlocks == 2) {
            philox_two((uint64_t)(m >> 2), step, a.keys, r[0], r[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) r[i] = philox((uint64_t)(m >> 2) + i, step, a.keys);
        }
        bool b[4 * kBlocks];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            b[4 * i] = r[i].x >= a.threshold;
            b[4 * i + 1] = r[i].y >= a.threshold;
            b[4 * i + 2] = r[i].z >= a.threshold;
            b[4 * i + 3] = r[i].w >= a.threshold;
        }
        if constexpr (SHIFTED) {
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 4 * kBlocks; ++i) bits |= (uint32_t)b[i] << i;
            bits >>= m & 3;
#pragma unroll
            for (int i = 0; i < E; ++i) k[i] = bits >> i & 1;
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) k[i] = b[i];
        }
    }
    __device__ __forceinline__ uint4 apply(uint4 v, float scale) const {
        alignas(16) T t[kVec<T>];
        memcpy(t, &v, 16);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            const float f = to_float(t[i]) * scale;
            t[i] = from_float<T>(k[i] ? f : 0.f);
        }
        memcpy(&v, t, 16);
        return v;
    }
};

// x one dense, aligned line and the mask as long: the whole pieces of it, `n` of them.
// Generator and memory take about the same time and have to overlap: many warps, with
// little between a load and the next.
template <typename T>
__global__ void __launch_bounds__(kDropThreads, 7) k_dropout_dense(const __grid_constant__ DropArgs a, int64_t n) {
    constexpr int kUnroll = 2;
    const uint64_t step = a.keys.at();
    const int64_t q0 = (int64_t)blockIdx.x * (kUnroll * kDropThreads) + threadIdx.x;
    const uint4 *x = (const uint4 *)a.x + q0;
    uint4 *y = (uint4 *)a.y + q0;
    uint4 v[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
        if (q0 + i * kDropThreads < n) v[i] = __ldcs(x + i * kDropThreads);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        if (q0 + i * kDropThreads >= n) return;
        Keep<T> keep;
        keep.template make<kPiece>(a, step, (q0 + i * kDropThreads) * kVec<T>);
        if (a.drop_all) v[i] = make_uint4(0, 0, 0, 0);
        __stcs(y + i * kDropThreads, keep.apply(v[i], a.scale));
    }
}

// LOCKED: the mask has `period` elements and y several times as many.  Where its pieces
// begin then depends on the factors that the period has.
template <typename T, bool LOCKED, int START>
__global__ void __launch_bounds__(kDropThreads) k_dropout_flat(const __grid_constant__ DropFlat f) {
    constexpr int E = kVec<T>, kUnroll = 1;
    const DropArgs &a = f.a;
    const uint64_t step = a.keys.at();
    const T *x = (const T *)a.x;
    T *y = (T *)a.y;
    const int64_t q0 = ((int64_t)blockIdx.x * kUnroll) * kDropThreads + threadIdx.x;
    uint4 v[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t e = (q0 + i * kDropThreads) * E;
        if (e >= f.n) continue;
        if (f.rows_joined && e + E <= f.n) {
            v[i] = load_vec<T>(x, e, f.n);
            continue;
        }
        int64_t row, plane;
        if (f.small) {
            row = f.row.quotient((uint32_t)e);
            plane = f.plane.quotient((uint32_t)row);
        } else {
            row = e / a.n3;
            plane = row / a.n2;
        }
        int64_t c = e - row * a.n3, r2 = row - plane * a.n2;
        // plane counts n1 or, locked, the repeats
        if (c + E <= a.n3) {
            v[i] = load_vec<T>(x + plane * a.x1 + r2 * a.x2, c, a.n3);
            continue;
        }
        alignas(16) T t[E];  // across a row's end, or the last
#pragma unroll
        for (int k = 0; k < E; ++k) {
            t[k] = e + k < f.n ? x[plane * a.x1 + r2 * a.x2 + c] : from_float<T>(0.f);
            if (++c == a.n3) {
                c = 0;
                if (++r2 == a.n2) r2 = 0, ++plane;
            }
        }
        memcpy(&v[i], t, 16);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t e = (q0 + i * kDropThreads) * E;
        if (e >= f.n) continue;
        const int64_t m = LOCKED ? (f.small ? (uint32_t)e % (uint32_t)f.period : e % f.period) : e;
        Keep<T> keep;
        keep.template make<START>(a, step, m);
        if (LOCKED && m + E > f.period) {  // the mask begins again, perhaps more than once
            for (int k = 0; k < E; ++k) {
                const int64_t mk = (m + k) % f.period;
                const uint4 r = philox((uint64_t)(mk >> 2), step, a.keys);
                const uint32_t w = (mk & 2) ? (mk & 1 ? r.w : r.z) : (mk & 1 ? r.y : r.x);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (j == k) keep.k[j] = w >= a.threshold;
            }
        }
        if (a.drop_all) v[i] = make_uint4(0, 0, 0, 0);
        const uint4 out = keep.apply(v[i], a.scale);
        if (e + E <= f.n) {
            __stcs((uint4 *)(y + e), out);
        } else {
            alignas(16) T t[E];
            memcpy(t, &out, 16);
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (e + k < f.n) y[e + k] = t[k];
        }
    }
}

// One mask for `rep` dense lines of n elements, n a multiple of E: it is made once
// and used for the lines of blockIdx.y's share.
template <typename T>
__global__ void __launch_bounds__(kDropThreads) k_dropout_lines(const __grid_constant__ DropFlat f, int lines) {
    constexpr int E = kVec<T>, kUnroll = 4;
    const DropArgs &a = f.a;
    const int64_t m = ((int64_t)blockIdx.x * kDropThreads + threadIdx.x) * E;
    if (m >= f.period) return;
    Keep<T> keep;
    keep.template make<kPiece>(a, a.keys.at(), m);
    const int64_t k0 = (int64_t)blockIdx.y * lines, k1 = k0 + lines < a.rep ? k0 + lines : a.rep;
    const T *x = (const T *)a.x + k0 * a.xr;
    T *y = (T *)a.y + k0 * f.period + m;
    for (int64_t k = k0; k < k1; k += kUnroll) {
        uint4 v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (k + i < k1) v[i] = load_vec<T>(x + i * a.xr, m, f.period);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (k + i < k1) {
                if (a.drop_all) v[i] = make_uint4(0, 0, 0, 0);
                __stcs((uint4 *)(y + i * f.period), keep.apply(v[i], a.scale));
            }
        x += kUnroll * a.xr;
        y += kUnroll * f.period;
    }
}

template <typename T> void launch_dropout(const DropArgs &a, cudaStream_t stream) {
    constexpr int E = kVec<T>;
    const int sms = device_sms();
    DropFlat f{};
    f.a = a;
    f.period = a.n1 * a.n2 * a.n3;
    f.n = f.period * a.rep;
    // y dense in the order of the mask and its repeats, and aligned; x's innermost axis dense
    const bool y_dense = (a.n3 == 1 || a.y3 == 1) && (a.n2 == 1 || a.y2 == a.n3) &&
                         (a.n1 == 1 || a.y1 == a.n2 * a.n3) && (a.rep == 1 || a.yr == f.period) &&
                         ((uintptr_t)a.y & 15) == 0;
    const bool x_line = a.n3 == 1 ? a.n2 * a.n1 * a.rep == 1 : a.x3 == 1;
    if (!y_dense || !x_line) {
        const int64_t want = (f.period / 4 + 255) / 256, most = 8 * (int64_t)sms;
        k_dropout<T><<<(int)(want < 1 ? 1 : want < most ? want : most), 256, 0, stream>>>(a);
        return;
    }
    const bool joined = (a.n2 == 1 || a.x2 == a.n3) && (a.n1 == 1 || a.x1 == a.n2 * a.n3);
    if (a.rep > 1 && joined && f.period % E == 0) {
        // a share of lines for each y of the grid: enough threads to fill the device twice
        const int64_t across = (f.period / E + kDropThreads - 1) / kDropThreads;
        int64_t shares = (16 * (int64_t)sms + across - 1) / across;
        if (shares > (a.rep + 3) / 4) shares = (a.rep + 3) / 4;
        if (shares > 65535) shares = 65535;
        const int64_t lines = (a.rep + shares - 1) / shares;
        const dim3 grid((unsigned)across, (unsigned)((a.rep + lines - 1) / lines));
        if (across < ((int64_t)1 << 31) && lines < ((int64_t)1 << 31)) {
            k_dropout_lines<T><<<grid, kDropThreads, 0, stream>>>(f, (int)lines);
            return;
        }
    }
    if (a.rep > 1) {
        // the repeats as the outermost axis
        f.a.n1 = a.rep;
        f.a.x1 = a.xr;
    }
    f.small = f.n < ((int64_t)1 << 31);
    f.rows_joined = joined && (a.rep == 1 || a.xr == f.period);
    if (f.small) {
        f.row = Divider::of((uint32_t)a.n3);
        f.plane = Divider::of((uint32_t)a.n2);
    }
    const int64_t pieces = (f.n + E - 1) / E;
    if (a.rep == 1 && f.rows_joined && ((uintptr_t)a.x & 15) == 0 && f.n % E == 0) {
        k_dropout_dense<T><<<(unsigned)((pieces + 2 * kDropThreads - 1) / (2 * kDropThreads)), kDropThreads, 0,
                             stream>>>(a, pieces);
        return;
    }
    const unsigned grid = (unsigned)((pieces + kDropThreads - 1) / kDropThreads);
    if (a.rep == 1)
        k_dropout_flat<T, false, kPiece><<<grid, kDropThreads, 0, stream>>>(f);
    else if (f.period % E == 0)
        k_dropout_flat<T, true, kPiece><<<grid, kDropThreads, 0, stream>>>(f);
    else if (f.period % 4 == 0)
        k_dropout_flat<T, true, kBlock><<<grid, kDropThreads, 0, stream>>>(f);
    else
        k_dropout_flat<T, true, kWithin><<<grid, kDropThreads, 0, stream>>>(f);
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" ck_status ck_dropout(const void *x, void *y, int64_t dtype, int64_t n0, int64_t n1,
                                int64_t n2, int64_t x0, int64_t x1, int64_t x2, int64_t y0,
                                int64_t y1, int64_t y2, int64_t locked, double p, uint64_t seed,
                                uint64_t step, const int64_t *step_dev, void *stream) {
    if (!known_dtype(dtype)) return fail(CK_ERR_INVALID_ARG, "dropout: unknown dtype %lld", (long long)dtype);
    if (!(p >= 0.0 && p <= 1.0)) return fail(CK_ERR_INVALID_ARG, "dropout: p must be in [0, 1]");
    if (n0 < 0 || n1 < 0 || n2 < 0) return fail(CK_ERR_INVALID_ARG, "dropout: negative size");
    if (n0 == 0 || n1 == 0 || n2 == 0) return CK_OK;
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (n0 > kMost / n1 || n0 * n1 > kMost / n2)
        return fail(CK_ERR_UNSUPPORTED, "dropout: more than 2^40 elements");
    if (!x || !y) return fail(CK_ERR_INVALID_ARG, "a required pointer is NULL");
    if ((n0 > 1 && y0 == 0) || (n1 > 1 && y1 == 0) || (n2 > 1 && y2 == 0))
        return fail(CK_ERR_INVALID_ARG, "dropout: elements of y share a place (a stride of 0)");
    if (!aligned(x, dtype_size(dtype)) || !aligned(y, dtype_size(dtype)) || !aligned(step_dev, 8))
        return fail(CK_ERR_INVALID_ARG, "dropout: a pointer is not aligned to its elements");
    DropArgs a{};
    a.x = x;
    a.y = y;
    a.rep = locked ? n0 : 1;
    a.n1 = locked ? 1 : n0;
    a.n2 = n1;
    a.n3 = n2;
    a.xr = a.x1 = x0;
    a.yr = a.y1 = y0;
    a.x2 = x1, a.x3 = x2, a.y2 = y1, a.y3 = y2;
    const double t = std::nearbyint(p * 4294967296.0);
    a.drop_all = t >= 4294967296.0;
    a.threshold = a.drop_all ? 0u : (uint32_t)t;
    a.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    a.keys = PhiloxKeys::of(seed, step, step_dev);
    with_dtype(dtype, [&](auto *tag) {
        launch_dropout<std::remove_pointer_t<decltype(tag)>>(a, (cudaStream_t)stream);
    });
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "k_dropout launch");
}
